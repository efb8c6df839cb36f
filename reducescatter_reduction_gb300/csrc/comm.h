// The communicator and the helpers that the host front ends share (ccl.cpp:
// the collectives; logits.cpp: the logit operators).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ccl.h"
#include "internal.h"

struct ccl_comm {
    int p = 0;
    int device = 0;
    int num_sms = 0;
    void *in[ccl::kMaxRanks] = {};
    void *out[ccl::kMaxRanks] = {};
    int sm_budget = 0;
    int variant = CCL_VARIANT_AUTO;
    size_t pipe_bytes = 0;
    unsigned *d_status = nullptr;   // device block: kCommStatusBytes of status, then the scratch of the loss sums
    bool has_custom = false;
    uint8_t custom[ccl::kMaxRanks * ccl::kMaxRanks] = {};
    ccl::Table table;               // last built table (one-entry cache)
    int table_sched = -1;
    bool table_valid = false;
    uint64_t launches = 0;
    char last[320] = "";
    long long wait_limit_ns = 2000000000LL;  // bounded device waits: 2 s
    int stall_test = 0;
};

namespace ccl {

// Set the message ccl_last_error() returns on this host thread; return st
// (cuda_fail: CCL_ERR_CUDA).
ccl_status_t fail(ccl_status_t st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
ccl_status_t cuda_fail(cudaError_t err, const char *what);
bool debug_on();   // CCL_DEBUG is set

constexpr const char *kDtypeName[] = {"f32", "f16", "bf16", "i32"};

// Restores the caller's current device when a call had to switch to the
// communicator's device.
struct DeviceGuard {
    int prev = -1;
    bool switched = false;
    cudaError_t err = cudaSuccess;
    explicit DeviceGuard(int dev)
    {
        err = cudaGetDevice(&prev);
        if (err == cudaSuccess && prev != dev) {
            err = cudaSetDevice(dev);
            switched = (err == cudaSuccess);
        }
    }
    ~DeviceGuard()
    {
        if (switched) cudaSetDevice(prev);
    }
};

// p balanced chunks, the first n % p one element larger.
inline void chunk_bounds(int p, uint64_t n, uint64_t *bounds)
{
    const uint64_t q = n / uint64_t(p), r = n % uint64_t(p);
    for (int c = 0; c <= p; ++c) {
        const uint64_t uc = uint64_t(c);
        bounds[c] = uc * q + (uc < r ? uc : r);
    }
}

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }

}  // namespace ccl
