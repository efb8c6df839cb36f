// What the host front ends of the operators share (logits.cpp, layers.cpp):
// argument checks, the launch record, the call's description.
#pragma once

#include <cstdio>

#include "comm.h"
#include "internal.h"

namespace ccl {

inline Range range_of(const void *p, uint64_t bytes)
{
    return {uintptr_t(p), p ? uintptr_t(p) + bytes : uintptr_t(p)};
}

inline ccl_status_t check_floats(const ccl_comm *c, int dtype, const char *what)
{
    if (!c) return fail(CCL_ERR_INVALID_ARG, "comm is NULL");
    if (dtype == CCL_I32) return fail(CCL_ERR_UNSUPPORTED, "%s needs a floating-point dtype", what);
    if (dtype < CCL_F32 || dtype > CCL_BF16) return fail(CCL_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    return CCL_OK;
}

inline ccl_status_t check_aligned(const void *p, size_t to, const char *name)
{
    if (uintptr_t(p) % to) return fail(CCL_ERR_INVALID_ARG, "%s is not aligned to its elements (%zu bytes)", name, to);
    return CCL_OK;
}

inline Launch make_launch(ccl_comm *c, int dtype, bool alias, void *stream)
{
    Launch L;
    L.p = c->p;
    L.dtype = dtype;
    for (int r = 0; r < c->p; ++r) {
        L.src[r] = c->in[r];
        L.dst[r] = c->out[r];
    }
    L.alias = alias;
    L.device = c->device;
    L.num_sms = c->num_sms;
    L.status = c->d_status;
    L.wait_limit_ns = c->wait_limit_ns;
    L.stall_test = c->stall_test;
    L.stream = static_cast<cudaStream_t>(stream);
    return L;
}

inline void describe_rows(ccl_comm *c)
{
    snprintf(c->last, sizeof c->last, "%s dtype=%s p=%d rows=%llu columns=%llu pass=%s grid=%d block=%d smem=%zu kernels=%d", c->call.kernel,
             kDtypeName[c->call_dtype], c->p, (unsigned long long)c->call_size[0], (unsigned long long)c->call_size[1], c->call_word, c->call.grid,
             c->call.block, c->call.smem, c->call.kernels);
}

inline ccl_status_t finish(ccl_comm *c, cudaError_t err, const LaunchInfo &info, int dtype, size_t rows, size_t cols, const char *what,
                           const char *pass)
{
    if (err == kTooManyPieces && info.kernels == 0)
        return fail(CCL_ERR_UNSUPPORTED, "%s: %zu rows of %zu columns over %d ranks are more than 2^31 - 1 pieces", what, rows, cols, c->p);
    c->launches += uint64_t(info.kernels);
    c->call = info;
    c->call_word = pass;
    c->call_dtype = dtype;
    c->call_size[0] = rows;
    c->call_size[1] = cols;
    c->describe = describe_rows;
    if (debug_on()) {
        describe_rows(c);
        fprintf(stderr, "[ccl] %s\n", c->last);
    }
    return err == cudaSuccess ? CCL_OK : cuda_fail(err, what);
}

}  // namespace ccl
