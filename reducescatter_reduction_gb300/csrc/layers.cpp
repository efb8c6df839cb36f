// Host front end of the operators around layers declared in include/ccl.h
// (norm with an 8-bit output, tokens by expert, gradient norm and clipping):
// argument and overlap checks, and the dispatch to their kernels.
#include "ccl.h"

#include <cuda_runtime.h>

#include <cfloat>
#include <new>

#include "front.h"
#include "spans.h"

using namespace ccl;

static ccl_status_t check_choices(const ccl_comm *c, size_t rows, size_t k, size_t capacity)
{
    const size_t most = 0x7fffffffull / size_t(c->p);
    if (k == 0 || k > 4096) return fail(CCL_ERR_INVALID_ARG, "k=%zu outside [1, 4096]", k);
    if (rows > most / k) return fail(CCL_ERR_INVALID_ARG, "ranks * rows * k above 2^31 - 1");
    if (capacity > most) return fail(CCL_ERR_INVALID_ARG, "ranks * capacity above 2^31 - 1: slots are 32-bit");
    return CCL_OK;
}

// ---------------------------------------------------------------------------
// Tokens by expert.
// ---------------------------------------------------------------------------

extern "C" ccl_status_t ccl_expert_sort(ccl_comm_t c, size_t rows, size_t experts, size_t k, const int32_t *const *expert_ids,
                                        const uint8_t *const *valid, size_t capacity, int32_t *const *slots, int32_t *offsets,
                                        void *stream)
{
    if (!c) return fail(CCL_ERR_INVALID_ARG, "comm is NULL");
    if (experts == 0) return fail(CCL_ERR_INVALID_ARG, "experts must be positive");
    if (experts > 4096) return fail(CCL_ERR_UNSUPPORTED, "experts=%zu above 4096", experts);
    ccl_status_t st = check_choices(c, rows, k, capacity);
    if (st != CCL_OK) return st;
    if (!offsets) return fail(CCL_ERR_INVALID_ARG, "offsets is NULL");
    if ((st = check_aligned(offsets, 4, "offsets")) != CCL_OK) return st;
    Spans s;
    s.add("offsets", -1, offsets, (experts + size_t(c->p)) * 4, true);
    if (rows) {
        if ((st = check_list(c, expert_ids, "expert_ids", 4)) != CCL_OK) return st;
        if (valid && (st = check_list(c, valid, "valid", 1)) != CCL_OK) return st;
        if ((st = check_list(c, slots, "slots", 4)) != CCL_OK) return st;
        for (int r = 0; r < c->p; ++r) {
            s.add("expert_ids", r, expert_ids[r], rows * k * 4, false);
            if (valid) s.add("valid", r, valid[r], rows, false);
            s.add("slots", r, slots[r], rows * k * 4, true);
        }
    }
    if ((st = check_spans(s.s, size_t(s.n))) != CCL_OK) return st;
    DeviceGuard g(c->device);
    if (g.err != cudaSuccess) return cuda_fail(g.err, "expert_sort");
    SortLaunch N;
    N.rows = rows;
    N.experts = uint32_t(experts);
    N.k = uint32_t(k);
    N.capacity = uint32_t(capacity);
    N.ids = expert_ids;
    N.valid = valid;
    N.slots = slots;
    N.offsets = offsets;
    N.cells = reinterpret_cast<int32_t *>(reinterpret_cast<char *>(c->d_status) + kSortOffset);
    LaunchInfo info;
    const cudaError_t err = launch_expert_sort(make_launch(c, CCL_I32, false, stream), N, &info);
    return finish(c, err, info, CCL_I32, rows, k, "expert_sort", "-");
}

static ccl_status_t expert_rows(ccl_comm *c, int op, int dtype, size_t rows, size_t hidden, size_t k, const int32_t *const *slots,
                                const float *const *weights, const void *const *experts, size_t capacity, float *const *dweights,
                                const char *what, void *stream)
{
    if (!c) return fail(CCL_ERR_INVALID_ARG, "comm is NULL");
    ccl_status_t st;
    if (op == ROWS_DISPATCH && dtype == CCL_I32) {
        if (weights) return fail(CCL_ERR_UNSUPPORTED, "%s: int32 rows have no weights", what);
    } else if ((st = check_floats(c, dtype, what)) != CCL_OK) {
        return st;
    }
    if ((st = check_choices(c, rows, k, capacity)) != CCL_OK) return st;
    const size_t es = elem_bytes(dtype);
    if (hidden == 0) return fail(CCL_ERR_INVALID_ARG, "hidden must be positive");
    if (hidden > (size_t(1) << 30)) return fail(CCL_ERR_UNSUPPORTED, "%s: hidden %zu above 2^30", what, hidden);   // columns are 32-bit
    const size_t most = rows > capacity ? rows : capacity;
    if (most && hidden > (SIZE_MAX / 4) / most / es) return fail(CCL_ERR_INVALID_ARG, "rows * hidden too large");
    if (rows == 0) return CCL_OK;
    if ((st = check_list(c, slots, "slots", 4)) != CCL_OK) return st;
    if (weights && (st = check_list(c, weights, "weights", 4)) != CCL_OK) return st;
    const size_t token_bytes = rows * hidden * es, expert_bytes = capacity * hidden * es;
    const bool to_tokens = op == ROWS_COMBINE;
    Spans s;
    uintptr_t bits = hidden * es;            // of every address and the row's bytes
    for (int r = 0; r < c->p; ++r) {
        const uintptr_t in = uintptr_t(c->in[r]), out = uintptr_t(c->out[r]);
        if (in % es || out % es)
            return fail(CCL_ERR_INVALID_ARG, "a buffer of rank %d is not aligned to its elements (%zu bytes)", r, es);
        bits |= in | out;
        s.add("the input of rank", r, c->in[r], to_tokens ? expert_bytes : token_bytes, false);
        s.add("the output of rank", r, c->out[r], to_tokens ? token_bytes : expert_bytes, true);
        s.add("slots", r, slots[r], rows * k * 4, false);
        if (weights) s.add("weights", r, weights[r], rows * k * 4, false);
    }
    if (op == ROWS_GRAD) {
        if ((st = check_list(c, experts, "expert_rows", es)) != CCL_OK) return st;
        if ((st = check_list(c, dweights, "dweights", 4)) != CCL_OK) return st;
        for (int r = 0; r < c->p; ++r) {
            bits |= uintptr_t(experts[r]);
            s.add("expert_rows", r, experts[r], expert_bytes, false);
            s.add("dweights", r, dweights[r], rows * k * 4, true);
        }
    }
    if ((st = check_spans(s.s, size_t(s.n))) != CCL_OK) return st;
    DeviceGuard g(c->device);
    if (g.err != cudaSuccess) return cuda_fail(g.err, what);
    Launch L = make_launch(c, dtype, false, stream);
    L.vec = bits % 16 == 0;
    RowsLaunch N;
    N.op = op;
    N.rows = rows;
    N.hidden = hidden;
    N.k = uint32_t(k);
    N.capacity = uint32_t(capacity);
    N.slots = slots;
    N.weights = weights;
    N.experts = experts;
    N.dweights = dweights;
    LaunchInfo info;
    const cudaError_t err = launch_expert_rows(L, N, &info);
    return finish(c, err, info, dtype, rows, hidden, what, "-");
}

extern "C" ccl_status_t ccl_expert_dispatch(ccl_comm_t c, ccl_dtype_t dtype, size_t rows, size_t hidden, size_t k,
                                            const int32_t *const *slots, const float *const *weights, size_t capacity, void *stream)
{
    return expert_rows(c, ROWS_DISPATCH, dtype, rows, hidden, k, slots, weights, nullptr, capacity, nullptr, "expert_dispatch", stream);
}

extern "C" ccl_status_t ccl_expert_combine(ccl_comm_t c, ccl_dtype_t dtype, size_t rows, size_t hidden, size_t k,
                                           const int32_t *const *slots, const float *const *weights, size_t capacity, void *stream)
{
    return expert_rows(c, ROWS_COMBINE, dtype, rows, hidden, k, slots, weights, nullptr, capacity, nullptr, "expert_combine", stream);
}

extern "C" ccl_status_t ccl_expert_combine_grad(ccl_comm_t c, ccl_dtype_t dtype, size_t rows, size_t hidden, size_t k,
                                                const int32_t *const *slots, const float *const *weights,
                                                const void *const *expert_rows_in, size_t capacity, float *const *dweights, void *stream)
{
    return expert_rows(c, ROWS_GRAD, dtype, rows, hidden, k, slots, weights, expert_rows_in, capacity, dweights, "expert_combine_grad",
                       stream);
}

// ---------------------------------------------------------------------------
// Gradients of many tensors.
// ---------------------------------------------------------------------------

static ccl_status_t grads(ccl_comm *c, size_t count, const ccl_tensor_t *tensors, bool clip, float max_norm, float *norm,
                          const char *what, void *stream)
{
    if (!c) return fail(CCL_ERR_INVALID_ARG, "comm is NULL");
    if (count && !tensors) return fail(CCL_ERR_INVALID_ARG, "tensors is NULL");
    if (count > 0x7fffffffull) return fail(CCL_ERR_INVALID_ARG, "count %zu above 2^31 - 1", count);
    if (!norm) return fail(CCL_ERR_INVALID_ARG, "norm is NULL");
    ccl_status_t st;
    if ((st = check_aligned(norm, 4, "norm")) != CCL_OK) return st;
    if (clip && !(max_norm >= 0.0f && max_norm <= FLT_MAX)) return fail(CCL_ERR_INVALID_ARG, "max_norm must be finite and >= 0");
    const Range at = range_of(norm, 8);
    // the stretches of memory that clipping reads and writes: tensors that follow one another are one; more than 64 go to the heap
    // (what is read in front and what is written behind it, as each often is in order already)
    Span few[64], *spans = few;
    size_t room = 32, reads = 0, writes = 0;
    uint64_t total = 0;
    st = CCL_OK;
    for (size_t i = 0; i < count && st == CCL_OK; ++i) {
        const ccl_tensor_t &t = tensors[i];
        if (t.dtype == CCL_I32) st = fail(CCL_ERR_UNSUPPORTED, "%s: tensor %zu needs a floating-point dtype", what, i);
        else if (t.dtype < CCL_F32 || t.dtype > CCL_BF16) st = fail(CCL_ERR_INVALID_ARG, "tensor %zu: unknown dtype %d", i, int(t.dtype));
        if (st != CCL_OK || t.n == 0) continue;
        const size_t es = elem_bytes(t.dtype);
        const Range in = range_of(t.in, t.n * es), out = clip ? range_of(t.out, t.n * es) : in;
        if (t.n > (uint64_t(1) << 40) || (total += t.n) > (uint64_t(1) << 40)) st = fail(CCL_ERR_INVALID_ARG, "more than 2^40 elements in all");
        else if (!in.lo || !out.lo) st = fail(CCL_ERR_INVALID_ARG, "tensor %zu is NULL", i);
        else if ((in.lo | out.lo) & (es - 1)) st = fail(CCL_ERR_INVALID_ARG, "tensor %zu is not aligned to its elements (%zu bytes)", i, es);
        else if (overlap(in, at) || overlap(out, at)) st = fail(CCL_ERR_INVALID_ARG, "norm overlaps tensor %zu", i);
        if (st != CCL_OK || !clip) continue;
        if (reads == room || writes == room) {
            Span *more = new (std::nothrow) Span[2 * count];
            if (!more) {
                st = fail(CCL_ERR_NOMEM, "host allocation failed");
                continue;
            }
            std::copy(spans, spans + reads, more);
            std::copy(spans + room, spans + room + writes, more + count);
            spans = more;
            room = count;
        }
        if (t.out != t.in) {
            if (reads && spans[reads - 1].at.hi == in.lo) spans[reads - 1].at.hi = in.hi;
            else spans[reads++] = {in, "the input of tensor", int(i), false};
        }
        Span *last = spans + room + writes;
        if (writes && last[-1].at.hi == out.lo) {
            last[-1].at.hi = out.hi;
        } else {
            *last = {out, "the output of tensor", int(i), true};
            ++writes;
        }
    }
    if (st == CCL_OK && writes) {
        std::copy(spans + room, spans + room + writes, spans + reads);
        st = check_spans(spans, reads + writes);
    }
    if (spans != few) delete[] spans;
    if (st != CCL_OK) return st;
    DeviceGuard g(c->device);
    if (g.err != cudaSuccess) return cuda_fail(g.err, what);
    GradLaunch N;
    N.count = count;
    N.tensors = tensors;
    N.clip = clip;
    N.max_norm = max_norm;
    N.norm = norm;
    N.scratch = reinterpret_cast<char *>(c->d_status) + kGradOffset;
    LaunchInfo info;
    const cudaError_t err = launch_grads(make_launch(c, CCL_F32, false, stream), N, &info);
    return finish(c, err, info, CCL_F32, count, total, what, "-");
}

extern "C" ccl_status_t ccl_grad_norm(ccl_comm_t c, size_t count, const ccl_tensor_t *tensors, float *norm, void *stream)
{
    return grads(c, count, tensors, false, 0.0f, norm, "grad_norm", stream);
}

extern "C" ccl_status_t ccl_grad_clip(ccl_comm_t c, size_t count, const ccl_tensor_t *tensors, float max_norm, float *norm, void *stream)
{
    return grads(c, count, tensors, true, max_norm, norm, "grad_clip", stream);
}
