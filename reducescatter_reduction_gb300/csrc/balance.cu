// The load-balance loss of a router over p data-parallel ranks: per-expert
// counts, the loss, and the gradient of the router's logits.
//
// With N the valid rows of all ranks, count_e the valid rows' choices of
// expert e over all ranks and p_t the softmax of row t:
//   loss = coef E sum_e f_e P_e,  f_e = count_e / (k N),  P_e = (1/N) sum_t p_te
//   dx_te = dloss p_te (a_e - sum_j p_tj a_j),  a_e = coef E count_e / (k N^2)
// Both need the counts only as a_e, so once the choices are counted one pass
// over the logits gives loss = sum_t sum_e p_te a_e and the gradient together.
// Differences of nearly equal a_e make the gradient: d_e = a_e - mean(a) is
// formed from the integer counts and rounded to fp32 once;
// p_te (d_e - sum_j p_tj d_j) is the same gradient, and the loss is
// mean(a) (rows with a softmax) + sum_t sum_e p_te d_e.
#include "async.cuh"
#include "logits.cuh"

#include <utility>

namespace ccl {

constexpr int kBalanceThreads = 256;
constexpr int kBalanceWarps = kBalanceThreads / 32;
constexpr int kCountThreads = 1024;
// Up to this many choices and counters in all, every CTA counts for itself
// instead of waiting for a counting kernel: one launch less.  Measured (8
// ranks, 64 bf16 experts, 6 choices; graph replay, us; counting here against
// the kernel): 3072 choices 7.6, 8.6; 8160 9.1, 9.1; 16320 11.7, 9.1.  Called
// one by one, the second launch costs the host about 3 us more.
constexpr uint64_t kCountHereIds = 8192;
constexpr uint64_t kCountHereCells = 4096;
// A row's exponentials are 2^(x c - m c) in one step up to this |m c|, with m
// its maximum and c = log2(e): the rounding of m c, at most 2^-5 there, is a
// factor of at most 1.022 that all of the row has and that divides out.
// Beyond, the difference x - m comes first: the rounding grows with m, and
// from some 10^9 on its power of two would be 0 or infinite.
constexpr float kOneStep = 1048576.0f;

template <int PM>
struct BalanceArgs {
    const void *in[PM];
    void *out[PM];
    const int32_t *ids[PM];
    const uint8_t *valid[PM];
    uint64_t rows;
    uint32_t p, experts, k;
    FastDiv by_k, by_choices, by_rows;   // choices per rank, rows per rank
    int pass, has_valid, count_here;
    double coef;
    const float *dloss;
    int32_t *counts, *tokens;      // the caller's
    int32_t *cells, *cell_tokens;  // where the counting kernel counts: the scratch, or the caller's own, zeroed
    float *loss;
    unsigned *ticket;
    double2 *partials;
    // checked build:
    unsigned *status;
    uint64_t held;                 // rows that every buffer and list has: `rows`, or one less where the debug hook wants the checks to fail
    uint32_t cell_room;            // counters that `cells` has
};

// The accesses that the checked build tests: to a rank buffer of elements of S bytes, a row's choices, its padding byte, a counter.
template <int PM>
__device__ __forceinline__ bool balance_holds(const BalanceArgs<PM> &a, const void *buf, uint32_t S, const void *at, uint32_t bytes)
{
    return !kBoundsCheck || in_buffer(at, bytes, buf, a.held * a.experts * S, a.status, kSiteBalance);
}
template <int PM>
__device__ __forceinline__ int balance_choice(const BalanceArgs<PM> &a, const int32_t *ids, uint64_t at)
{
    return in_bounds(at < a.held * a.k, a.status, kSiteBalance, at) ? ids[at] : -1;
}
template <int PM>
__device__ __forceinline__ bool balance_valid(const BalanceArgs<PM> &a, const uint8_t *valid, uint64_t row)
{
    return in_bounds(row < a.held, a.status, kSiteBalance, row) && valid[row];
}
template <int PM>
__device__ __forceinline__ bool balance_cell(const BalanceArgs<PM> &a, uint64_t cell)
{
    return in_bounds(cell < a.cell_room, a.status, kSiteBalance, cell);
}

// Counts the choices and valid rows of all ranks into cells, which are zero.
// A CTA counts in shared memory first: integer atomics, so any order gives
// the same counts.  Bound by latency and the shared-memory atomics: 1 Mi
// choices of 256 experts add 8 us to the call.  The cells are the
// communicator's scratch, left at zero by the call's last CTA; with a memset
// of the caller's counters instead, 8 x 16384 x 256 bf16 took 37.4 us, not
// 32.6 (what calls do whose p * experts the scratch does not hold).
template <int PM>
__global__ void __launch_bounds__(kCountThreads) balance_count_kernel(const __grid_constant__ BalanceArgs<PM> a)
{
    extern __shared__ int hist[];
    constexpr int BATCH = 8;
    const uint32_t r = blockIdx.y;
    for (uint32_t e = threadIdx.x; e < a.experts; e += kCountThreads) hist[e] = 0;
    grid_dependency_wait();
    grid_dependents_launch();
    __syncthreads();
    const uint64_t first = uint64_t(blockIdx.x) * kCountThreads + threadIdx.x, stride = uint64_t(gridDim.x) * kCountThreads;
    const uint64_t n = a.rows * a.k;
    const int32_t *ids = a.ids[r];
    for (uint64_t j = first; j < n; j += BATCH * stride) {
        int id[BATCH];
        bool on[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const uint64_t at = j + b * stride;
            id[b] = at < n ? balance_choice(a, ids, at) : -1;
            on[b] = at < n && (!a.has_valid || balance_valid(a, a.valid[r], div_by(uint32_t(at), a.by_k)));
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
            if (on[b] && uint32_t(id[b]) < a.experts) atomicAdd(&hist[id[b]], 1);
    }
    if (a.has_valid) {
        int rows = 0;
        for (uint64_t t = first; t < a.rows; t += stride) rows += balance_valid(a, a.valid[r], t);
        rows = __reduce_add_sync(0xffffffffu, rows);
        if (threadIdx.x % 32 == 0 && rows) atomicAdd(&a.cell_tokens[r], rows);
    } else if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.cell_tokens[r] = int(a.rows);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.experts; e += kCountThreads)
        if (hist[e] && balance_cell(a, uint64_t(r) * a.experts + e)) atomicAdd(&a.cells[uint64_t(r) * a.experts + e], hist[e]);
}

// d_e into shared memory; returns where mean(a) is: in fp64, as the loss is
// next to nothing but n times it where the experts are balanced.  hist: p *
// experts counters and p row counts where the CTA counts for itself.
template <int PM>
__device__ __forceinline__ const double *balance_coefficients(const BalanceArgs<PM> &a, float *d_s, int *hist)
{
    __shared__ unsigned long long parts[2][kBalanceWarps];   // valid rows, choices
    const uint32_t E = a.experts;
    const int32_t *cells = a.cells, *tokens = a.cell_tokens;
    if (a.count_here) {
        int *rows_s = hist + a.p * E;
        for (uint32_t i = threadIdx.x; i < a.p * E + a.p; i += kBalanceThreads) hist[i] = 0;
        __syncthreads();
        constexpr int BATCH = 8;
        const uint32_t rows = uint32_t(a.rows), n = rows * a.k, all = a.p * n;
        for (uint32_t i = threadIdx.x; i < all; i += BATCH * kBalanceThreads) {
            int id[BATCH];
            uint32_t rank[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const uint32_t at = i + b * kBalanceThreads;
                id[b] = -1;
                if (at >= all) continue;
                rank[b] = div_by(at, a.by_choices);
                const uint32_t j = at - rank[b] * n;
                id[b] = balance_choice(a, a.ids[rank[b]], j);
                if (a.has_valid && !balance_valid(a, a.valid[rank[b]], div_by(j, a.by_k))) id[b] = -1;
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
                if (uint32_t(id[b]) < E) atomicAdd(&hist[rank[b] * E + id[b]], 1);
        }
        if (a.has_valid) {
            for (uint32_t i = threadIdx.x; i < a.p * rows; i += kBalanceThreads) {
                const uint32_t rank = div_by(i, a.by_rows);
                if (balance_valid(a, a.valid[rank], i - rank * rows)) atomicAdd(&rows_s[rank], 1);
            }
        } else {
            for (uint32_t r = threadIdx.x; r < a.p; r += kBalanceThreads) rows_s[r] = int(rows);
        }
        cells = hist;
        tokens = rows_s;
    }
    __syncthreads();
    auto count_of = [&](uint32_t r, uint32_t e) -> unsigned {
        const uint64_t cell = uint64_t(r) * E + e;
        return balance_cell(a, cell) ? unsigned(cells[cell]) : 0u;
    };
    // sums of integers: any order gives the same
    const bool writes = a.cells != a.counts && blockIdx.x == 0 && blockIdx.y == 0;
    unsigned long long rows = 0, mine = 0, total = 0;    // total: of this thread's first expert
    for (uint32_t r = threadIdx.x; r < a.p; r += kBalanceThreads) {
        rows += unsigned(tokens[r]);
        if (writes) a.tokens[r] = tokens[r];
    }
    for (uint32_t e = threadIdx.x; e < E; e += kBalanceThreads) {
        unsigned long long t = 0;
#pragma unroll 8
        for (uint32_t r = 0; r < a.p; ++r) t += count_of(r, e);
        if (writes)
            for (uint32_t r = 0; r < a.p; ++r) a.counts[uint64_t(r) * E + e] = int(count_of(r, e));
        if (e == threadIdx.x) total = t;
        mine += t;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        rows += __shfl_xor_sync(0xffffffffu, rows, o);
        mine += __shfl_xor_sync(0xffffffffu, mine, o);
    }
    if (threadIdx.x % 32 == 0) {
        parts[0][threadIdx.x / 32] = rows;
        parts[1][threadIdx.x / 32] = mine;
    }
    __syncthreads();
    unsigned long long all_rows = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kBalanceWarps; ++w) {
        all_rows += parts[0][w];
        all += parts[1][w];
    }
    // a_e = count_e scale, d_e = (E count_e - sum) scale / E.  The difference is exact in 64-bit integers; it and scale / E are
    // taken as a sum of two fp32 values each, so that d_e is rounded once.  scale / E = coef / (k n^2) comes by products whose
    // roundings are kept (fma), a quotient and what it leaves: fp64, which this GPU does slowly, is for the mean alone.
    __shared__ float scale_s[2];
    __shared__ double mean_s;
    if (threadIdx.x == 0) {
        const float k = float(a.k), n = float(all_rows), n_rest = float((long long)(all_rows - (unsigned long long)n));
        const float nn = __fmul_rn(n, n), nn_rest = fmaf(n, n, -nn) + 2.0f * n * n_rest;
        const float by = __fmul_rn(nn, k), by_rest = fmaf(nn, k, -by) + nn_rest * k;
        const float coef = float(a.coef), hi = all_rows ? __fdiv_rn(coef, by) : 0.0f;
        scale_s[0] = hi;
        scale_s[1] = all_rows ? __fdiv_rn(fmaf(-hi, by_rest, fmaf(-hi, by, coef)), by) : 0.0f;
    }
    __syncthreads();
    const float per = scale_s[0], per_rest = scale_s[1];
    const long long sum = (long long)all;
    for (uint32_t e = threadIdx.x; e < E; e += kBalanceThreads) {
        unsigned long long t = total;
        if (e != threadIdx.x) {
            t = 0;
            for (uint32_t r = 0; r < a.p; ++r) t += count_of(r, e);
        }
        const long long off = (long long)(t * E) - sum;
        const float hi = float(off), lo = fabsf(hi) < 16777216.0f ? 0.0f : float(off - (long long)hi);
        d_s[e] = fmaf(hi, per, fmaf(hi, per_rest, lo * per));
    }
    __syncthreads();
    if (threadIdx.x == kBalanceThreads - 1 && a.pass != CCL_PASS_BACKWARD) {    // (read at the end, behind other barriers)
        const double n = double(all_rows);
        mean_s = all_rows ? double(all) * (a.coef / (double(a.k) * n * n)) : 0.0;
    }
    return &mean_s;
}

// The CTAs' sums: each leaves its pair, the last one adds the pairs in the
// order of the CTAs, writes the loss and leaves the scratch at zero.
template <int PM>
__device__ __forceinline__ void balance_finish(const BalanceArgs<PM> &a, float lean, int live, const double *mean)
{
    __shared__ double red[2][kBalanceWarps];
    __shared__ bool last;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lean += __shfl_xor_sync(0xffffffffu, lean, o);
    live = __reduce_add_sync(0xffffffffu, live);
    double s, c;
    if (lane == 0) {
        red[0][warp] = lean;
        red[1][warp] = live;
    }
    __syncthreads();
    const unsigned grid = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
    if (threadIdx.x == 0) {
        s = c = 0.0;
        for (int w = 0; w < kBalanceWarps; ++w) {
            s += red[0][w];
            c += red[1][w];
        }
        if (in_bounds(me < kMaxPartials, a.status, kSiteBalance, me)) a.partials[me] = make_double2(s, c);
        __threadfence();
        last = atomicAdd(a.ticket, 1u) == grid - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (a.cells != a.counts && !a.count_here) {
        for (uint32_t i = threadIdx.x; i < a.p * a.experts; i += kBalanceThreads)
            if (balance_cell(a, i)) a.cells[i] = 0;
        for (uint32_t r = threadIdx.x; r < a.p; r += kBalanceThreads) a.cell_tokens[r] = 0;
    }
    s = c = 0.0;
    for (unsigned i = threadIdx.x; i < grid; i += kBalanceThreads) {
        const double2 v = __ldcg(&a.partials[i]);
        s += v.x;
        c += v.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        c += __shfl_xor_sync(0xffffffffu, c, o);
    }
    if (lane == 0) {
        red[0][warp] = s;
        red[1][warp] = c;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        s = c = 0.0;
        for (int w = 0; w < kBalanceWarps; ++w) {
            s += red[0][w];
            c += red[1][w];
        }
        *a.loss = float(s + c * *mean);
        *a.ticket = 0;
    }
}

// L lanes of a warp take a row, 16-byte groups l, l + L, ... of it; NV groups
// a lane hold the whole row, so the logits are read once and the next row's
// are on their way meanwhile; L is as small as holds the row, for fewer
// shuffles.  Bound by memory and about 12 us of launches, counting and the
// last CTA's sum: 8 x 16384 x 256 bf16, loss and gradient, 32.9 us (4.2 TB/s
// in all); f32, 4 x 65536 x 128, the loss, 30.9 us (4.4 TB/s).
template <typename T, int PM, int L, int NV>
__global__ void __launch_bounds__(kBalanceThreads, NV * Traits<T>::VEC > 16 ? 2 : NV > 2 ? 3 : 4) balance_kernel(const __grid_constant__ BalanceArgs<PM> a)
{
    using Tr = Traits<T>;
    using Gr = Group<T>;
    constexpr int VEC = Tr::VEC, S = 16 / VEC, RPW = 32 / L, PAIRS = Gr::PAIRS;
    extern __shared__ float d_s[];
    const uint32_t E = a.experts, r = blockIdx.y;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, l = lane % L;
    const bool fwd = a.pass & CCL_PASS_FORWARD, bwd = a.pass & CCL_PASS_BACKWARD;
    const uint8_t *valid = a.has_valid ? a.valid[r] : nullptr;
    const uint64_t stride = uint64_t(gridDim.x) * kBalanceWarps * RPW;
    const uint64_t row_bytes = uint64_t(E) * S, hop = stride * row_bytes;
    uint64_t t = (uint64_t(blockIdx.x) * kBalanceWarps + warp) * RPW + lane / L;   // this lane's row
    const char *at = static_cast<const char *>(a.in[r]) + t * row_bytes + l * 16;
    const ptrdiff_t to_out = static_cast<char *>(a.out[r]) - static_cast<const char *>(a.in[r]);
    bool has[NV];       // group n of a row is this lane's
#pragma unroll
    for (int n = 0; n < NV; ++n) has[n] = uint32_t((n * L + l) * VEC) < E;
    bool on = false;
    uint4 raw[NV];
    auto fetch = [&](uint64_t row, const char *from) {
        const bool in = row < a.rows;
        on = in && (!valid || balance_valid(a, valid, row));
#pragma unroll
        for (int n = 0; n < NV; ++n)
            raw[n] = in && has[n] && balance_holds(a, a.in[r], S, from + n * (L * 16), 16) ? ld_coherent_v4(from + n * (L * 16)) : lowest_group<T>();
    };
    grid_dependency_wait();
    grid_dependents_launch();
    fetch(t, at);
    const double *mean = balance_coefficients(a, d_s, reinterpret_cast<int *>(d_s + E));
    Pair d[NV * PAIRS];
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const uint32_t col = (n * L + l) * VEC + 2 * i;
            d[n * PAIRS + i] = {col < E ? d_s[col] : 0.0f, col + 1 < E ? d_s[col + 1] : 0.0f};
        }
    const float up = bwd && a.dloss ? *a.dloss : 1.0f;
    float lean_sum = 0.0f;
    int live = 0;
    const uint64_t last = a.rows + lane / L;     // rows of a warp end together: its lanes leave together
    for (; t < last; t += stride, at += hop) {
        uint4 v[NV];
#pragma unroll
        for (int n = 0; n < NV; ++n) v[n] = on ? raw[n] : lowest_group<T>();   // padding: p = 0, whatever it holds
        fetch(t + stride, at + hop);
        typename Gr::Max gm = Gr::lowest();
#pragma unroll
        for (int n = 0; n < NV; ++n) gm = Gr::max(gm, v[n]);
        float m = Gr::value(gm);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = finite_max(m);
        Pair x[NV * PAIRS], sum = {0.0f, 0.0f}, dot = {0.0f, 0.0f};
        const float mc = m * kLog2e;
        if (__all_sync(0xffffffffu, fabsf(mc) < kOneStep)) {
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) x[n * PAIRS + i] = ex2(fma(Gr::pair(v[n], i), Pair{kLog2e, kLog2e}, Pair{-mc, -mc}));
        } else {
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) x[n * PAIRS + i] = ex2((Gr::pair(v[n], i) + Pair{-m, -m}) * Pair{kLog2e, kLog2e});
        }
#pragma unroll
        for (int i = 0; i < NV * PAIRS; ++i) {
            sum = sum + x[i];
            dot = fma(x[i], d[i], dot);
        }
        float s = sum.x + sum.y, w = dot.x + dot.y;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            const float s2 = __shfl_xor_sync(0xffffffffu, s, o), w2 = __shfl_xor_sync(0xffffffffu, w, o);
            s += s2;
            w += w2;
        }
        const float inv = s == 0.0f ? 0.0f : 1.0f / s;    // a row of nothing but -inf has no softmax: p = 0
        const float lean = w * inv;
        if (l == 0 && s != 0.0f) {
            lean_sum += lean;
            ++live;
        }
        if (bwd && t < a.rows) {
            const Pair g = {inv * up, inv * up}, off = {-lean, -lean};
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                if (!has[n] || !balance_holds(a, a.out[r], S, at + to_out + n * (L * 16), 16)) continue;
                Pair f[PAIRS];
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) f[i] = (x[n * PAIRS + i] * (d[n * PAIRS + i] + off)) * g;
                st_stream_v4(const_cast<char *>(at) + to_out + n * (L * 16), Gr::pack(f));
            }
        }
    }
    if (fwd) balance_finish(a, lean_sum, live, mean);
}

// Rows of up to 1024 experts that are not whole, aligned 16-byte groups.  A
// warp takes 32 / L rows at a time: they are consecutive in memory, so it
// brings the groups that hold them into shared memory asynchronously, STAGES
// - 1 steps ahead, and its lanes read their elements l, l + L, ... from there;
// the gradient goes back the same way, whole groups and a few edge elements.
// Bound by instructions, element by element: 8 x 60000 x 60 bf16 with four
// choices 44 us, 8 x 20000 x 203 51, 8 x 400000 x 9 73, 8 x 6000 x 700 47.  (At
// the time, a warp per row without the stages: 152, 87, 721, 71 for 61, 68, 77
// and 51; four CTAs per SM for three: 51, 59, 70 for 50, 55, 70.)
// Where the rows are aligned groups balance_kernel is the faster: 8 x 65536 x
// 64 bf16 32 against 76 us, 8 x 32768 x 128 f32 50 against 57.
template <int NE>
constexpr int kOddStages = NE > 16 ? 2 : 3;
template <int NE>
constexpr int kOddCtas = NE > 16 ? 2 : 3;     // per SM

// f(0) ... f(N - 1), each with its number as a constant
template <int N, typename F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f)
{
    each_of<N>(f, std::make_integer_sequence<int, N>{});
}

constexpr uint32_t kOddSlack = 256;           // bytes that reads past the last row may reach into
// bytes of a step's groups, wherever in a group its rows begin
__host__ __device__ inline uint32_t odd_span(uint32_t rows, uint32_t row_bytes) { return (rows * row_bytes + 30) / 16 * 16; }

// One element from or to shared memory, OFF bytes beyond addr.
template <typename T, int OFF>
__device__ __forceinline__ float lds_element(uint32_t addr)
{
    uint32_t v;
    if constexpr (Traits<T>::VEC == 4) {
        asm volatile("ld.shared.u32 %0, [%1+%2];" : "=r"(v) : "r"(addr), "n"(OFF) : "memory");
        return __uint_as_float(v);
    } else {
        asm volatile("ld.shared.u16 %0, [%1+%2];" : "=r"(v) : "r"(addr), "n"(OFF) : "memory");
        return Group<T>::pair(make_uint4(v, 0, 0, 0), 0).x;
    }
}

// The pair's elements, OFF and NEXT bytes beyond addr; the second only if `both`.
template <typename T, int OFF, int NEXT>
__device__ __forceinline__ void sts_pair(uint32_t addr, Pair v, bool first, bool both)
{
    if constexpr (Traits<T>::VEC == 4) {
        if (first) asm volatile("st.shared.f32 [%0+%1], %2;" ::"r"(addr), "n"(OFF), "f"(v.x) : "memory");
        if (both) asm volatile("st.shared.f32 [%0+%1], %2;" ::"r"(addr), "n"(NEXT), "f"(v.y) : "memory");
    } else {
        const uint32_t w = Traits<T>::pack2(v.x, v.y);
        if (first) asm volatile("st.shared.u16 [%0+%1], %2;" ::"r"(addr), "n"(OFF), "r"(w) : "memory");
        if (both) asm volatile("st.shared.u16 [%0+%1], %2;" ::"r"(addr), "n"(NEXT), "r"(w >> 16) : "memory");
    }
}

template <typename T, int PM, int L, int NE>
__global__ void __launch_bounds__(kBalanceThreads, kOddCtas<NE>) balance_odd_kernel(const __grid_constant__ BalanceArgs<PM> a)
{
    using Tr = Traits<T>;
    constexpr int S = 16 / Tr::VEC, RPW = 32 / L, PAIRS = NE / 2, STAGES = kOddStages<NE>;
    extern __shared__ __align__(16) unsigned char stages_s[];
    const uint32_t E = a.experts, r = blockIdx.y, row_bytes = E * S, span = odd_span(RPW, row_bytes);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, l = lane % L, mine = lane / L;
    unsigned char *in_s = stages_s + warp * (STAGES + 1) * span, *out_s = in_s + STAGES * span;
    // a row of -inf, which is what a padding row is read as
    unsigned char *low_s = stages_s + kBalanceWarps * (STAGES + 1) * span;
    float *d_s = reinterpret_cast<float *>(low_s + (row_bytes + 15) / 16 * 16 + kOddSlack);
    for (uint32_t e = threadIdx.x; e < E; e += kBalanceThreads) Tr::store1(low_s, e, -INFINITY);
    const bool fwd = a.pass & CCL_PASS_FORWARD, bwd = a.pass & CCL_PASS_BACKWARD;
    const uint8_t *valid = a.has_valid ? a.valid[r] : nullptr;
    const uint64_t stride = uint64_t(gridDim.x) * kBalanceWarps * RPW;
    const uintptr_t in = uintptr_t(a.in[r]), in_end = in + a.rows * row_bytes, out = uintptr_t(a.out[r]), out_end = out + a.rows * row_bytes;
    uint64_t t = (uint64_t(blockIdx.x) * kBalanceWarps + warp) * RPW;    // the warp's first row
    auto fetch = [&](uint64_t row, uint32_t stage) {
        if (row < a.rows) {
            const uintptr_t b0 = in + row * row_bytes, b1 = min(b0 + RPW * row_bytes, in_end), lo = b0 & ~uintptr_t(15);
            unsigned char *to = in_s + stage * span;
            const uint32_t n = uint32_t(b1 - lo), to32 = smem_addr(to);
            if (lo >= in && lo + (n + 15) / 16 * 16 <= in_end) {
#pragma unroll 1
                for (uint32_t g = lane * 16; g < n; g += 512)
                    if (in_bounds(g + 16 <= span, a.status, kSiteBalance, row) && balance_holds(a, a.in[r], S, reinterpret_cast<const void *>(lo + g), 16))
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to32 + g), "l"(lo + g) : "memory");
            } else {      // the first or last group of the buffer is not all of it
#pragma unroll 1
                for (uint32_t g = lane * S; g < n; g += 32 * S)
                    if (lo + g >= in && in_bounds(g + S <= span, a.status, kSiteBalance, row) &&
                        balance_holds(a, a.in[r], S, reinterpret_cast<const void *>(lo + g), S))
                        Tr::store1(to + g, 0, Tr::load1(reinterpret_cast<const void *>(lo + g), 0));
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    grid_dependency_wait();
    grid_dependents_launch();
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(t + i * stride, i);
    auto is_on = [&](uint64_t row) { return row < a.rows && (!valid || balance_valid(a, valid, row)); };
    bool coming = is_on(t + mine);
    const double *mean = balance_coefficients(a, d_s, reinterpret_cast<int *>(d_s + E));
    Pair d[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        const uint32_t e = 2 * i * L + l;
        d[i] = {e < E ? d_s[e] : 0.0f, e + L < E ? d_s[e + L] : 0.0f};
    }
    const float up = bwd && a.dloss ? *a.dloss : 1.0f;
    float lean_sum = 0.0f;
    int live = 0;
    // pair i is nobody's; L is the smallest that holds a row, so only the upper half can be
    auto beyond = [&](int i) { return (L == 1 || i >= PAIRS / 2) && 2 * i * L >= int(E); };
    uint32_t stage = 0;
    for (; t < a.rows; t += stride) {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
        __syncwarp();
        fetch(t + (STAGES - 1) * stride, stage == 0 ? STAGES - 1 : stage - 1);
        const bool on = coming;
        coming = is_on(t + stride + mine);
        const uintptr_t b0 = in + t * row_bytes, o0 = out + t * row_bytes;
        const uint32_t from = smem_addr(on ? in_s + stage * span + b0 % 16 + mine * row_bytes : low_s) + l * S;
        stage = stage + 1 == STAGES ? 0 : stage + 1;
        Pair x[PAIRS];
        float m = -INFINITY;
        each<PAIRS>([&](auto I) {
            constexpr int i = decltype(I)::value;
            x[i] = {-INFINITY, -INFINITY};
            if (beyond(i)) return;
            // reads past the row, up to 2 L elements, are of shared memory all the same
            const float v0 = lds_element<T, 2 * i * L * S>(from), v1 = lds_element<T, (2 * i + 1) * L * S>(from);
            x[i] = {v0, v1};
            if ((L == 1 || i >= PAIRS / 2 - 1) && (2 * i + 2) * L > E) {
                if (2 * i * L + l >= E) x[i].x = -INFINITY;
                if ((2 * i + 1) * L + l >= E) x[i].y = -INFINITY;
            }
            m = fmaxf(m, fmaxf(x[i].x, x[i].y));
        });
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = finite_max(m);
        Pair sum = {0.0f, 0.0f}, dot = {0.0f, 0.0f};
        const float mc = m * kLog2e;             // (as in balance_kernel)
        if (__all_sync(0xffffffffu, fabsf(mc) < kOneStep)) {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i)
                if (!beyond(i)) x[i] = ex2(fma(x[i], Pair{kLog2e, kLog2e}, Pair{-mc, -mc}));
        } else {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i)
                if (!beyond(i)) x[i] = ex2((x[i] + Pair{-m, -m}) * Pair{kLog2e, kLog2e});
        }
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            if (beyond(i)) continue;
            sum = sum + x[i];
            dot = fma(x[i], d[i], dot);
        }
        float s = sum.x + sum.y, w = dot.x + dot.y;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            const float s2 = __shfl_xor_sync(0xffffffffu, s, o), w2 = __shfl_xor_sync(0xffffffffu, w, o);
            s += s2;
            w += w2;
        }
        const float inv = s == 0.0f ? 0.0f : 1.0f / s;
        const float lean = w * inv;
        if (l == 0 && s != 0.0f) {
            lean_sum += lean;
            ++live;
        }
        if (bwd) {
            const Pair g = {inv * up, inv * up}, off = {-lean, -lean};
            const uint32_t to = smem_addr(out_s) + uint32_t(o0 % 16) + mine * row_bytes + l * S;
            each<PAIRS>([&](auto I) {
                constexpr int i = decltype(I)::value;
                if (beyond(i)) return;
                const bool full = (L > 1 && i < PAIRS / 2 - 1) || (2 * i + 2) * L <= E;
                sts_pair<T, 2 * i * L * S, (2 * i + 1) * L * S>(to, (x[i] * (d[i] + off)) * g, full || 2 * i * L + l < E,
                                                               full || (2 * i + 1) * L + l < E);
            });
            __syncwarp();
            const uintptr_t o1 = min(o0 + RPW * row_bytes, out_end), low = o0 & ~uintptr_t(15);
            const uintptr_t first = (o0 + 15) & ~uintptr_t(15), last = o1 & ~uintptr_t(15), head = min(first, o1), tail = max(last, head);
            if (!in_bounds(o1 - low <= span, a.status, kSiteBalance, t)) continue;
            const uint32_t skip = uint32_t(first - low), whole = last > first ? uint32_t(last - first) : 0u, out32 = smem_addr(out_s) + skip;
#pragma unroll 1
            for (uint32_t g = lane * 16; g < whole; g += 512)
                if (balance_holds(a, a.out[r], S, reinterpret_cast<const void *>(first + g), 16))
                    st_stream_v4(reinterpret_cast<void *>(first + g), lds_v4(out32 + g));
            const uintptr_t edge = lane < 8 ? o0 + lane * S : tail + (lane - 8) * S;     // at most seven before, and seven after
            if (lane < 16 && edge < (lane < 8 ? head : o1) && balance_holds(a, a.out[r], S, reinterpret_cast<const void *>(edge), S))
                Tr::store1(reinterpret_cast<void *>(edge), 0, Tr::load1(out_s + (edge - low), 0));
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (fwd) balance_finish(a, lean_sum, live, mean);
}

// More than 1024 experts: a warp per row, element by element, the row read
// once per step (the later reads from cache).  8 x 2048 x 2048 bf16: 89 us.
template <typename T, int PM>
__global__ void __launch_bounds__(kBalanceThreads) balance_any_kernel(const __grid_constant__ BalanceArgs<PM> a)
{
    using Tr = Traits<T>;
    extern __shared__ float d_s[];
    const uint32_t E = a.experts, r = blockIdx.y;
    grid_dependency_wait();
    grid_dependents_launch();
    const double *mean = balance_coefficients(a, d_s, reinterpret_cast<int *>(d_s + E));
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const bool fwd = a.pass & CCL_PASS_FORWARD, bwd = a.pass & CCL_PASS_BACKWARD;
    const float up = bwd && a.dloss ? *a.dloss : 1.0f;
    float lean_sum = 0.0f;
    int live = 0;
    for (uint64_t t = uint64_t(blockIdx.x) * kBalanceWarps + warp; t < a.rows; t += uint64_t(gridDim.x) * kBalanceWarps) {
        const uint64_t at = t * E;
        constexpr uint32_t S = 16 / Tr::VEC;
        auto load = [&](uint32_t e) -> float {
            return balance_holds(a, a.in[r], S, static_cast<const char *>(a.in[r]) + (at + e) * S, S) ? Tr::load1(a.in[r], at + e) : -INFINITY;
        };
        auto store = [&](uint32_t e, float v) {
            if (balance_holds(a, a.out[r], S, static_cast<const char *>(a.out[r]) + (at + e) * S, S)) Tr::store1(a.out[r], at + e, v);
        };
        const bool valid = !a.has_valid || balance_valid(a, a.valid[r], t);
        if (!valid) {
            if (bwd)
                for (uint32_t e = lane; e < E; e += 32) store(e, 0.0f);
            continue;
        }
        float m = -INFINITY;
        for (uint32_t e = lane; e < E; e += 32) m = fmaxf(m, load(e));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = m == -INFINITY ? 0.0f : m;
        float s = 0.0f, dot = 0.0f;
        for (uint32_t e = lane; e < E; e += 32) {
            const float v = ex2((load(e) - m) * kLog2e);
            s += v;
            dot = fmaf(v, d_s[e], dot);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        const float inv = s == 0.0f ? 0.0f : 1.0f / s;
        const float lean = dot * inv;
        if (lane == 0 && s != 0.0f) {
            lean_sum += lean;
            ++live;
        }
        if (bwd) {
            const float g = inv * up;
            for (uint32_t e = lane; e < E; e += 32) {
                const float v = ex2((load(e) - m) * kLog2e);
                store(e, v * (d_s[e] - lean) * g);
            }
        }
    }
    if (fwd) balance_finish(a, lean_sum, live, mean);
}

// The most shared memory: rows of the lanes' elements, an expert's coefficient, and a count per cell.
template <typename T, int PM, int L, int NE>
static cudaError_t odd_kernel(int device, void (**kern)(BalanceArgs<PM>))
{
    constexpr uint32_t most = L * NE;
    static std::atomic<unsigned long long> done{0};
    *kern = balance_odd_kernel<T, PM, L, NE>;
    return allow_dynamic_smem(*kern, kBalanceWarps * (kOddStages<NE> + 1) * size_t(odd_span(32 / L, most * (16 / Traits<T>::VEC))) + kOddSlack + most * 8 +
                                         (kCountHereCells + PM) * 4, device, done);
}

template <typename T, int PM>
static cudaError_t balance_shape(const Launch &L, const BalanceLaunch &N, LaunchInfo *info)
{
    constexpr int VEC = Traits<T>::VEC, NV = 16 / VEC;
    BalanceArgs<PM> a;
    bool vec = N.experts % VEC == 0;
    const bool bwd = N.pass & CCL_PASS_BACKWARD, fwd = N.pass & CCL_PASS_FORWARD;
    for (int r = 0; r < L.p; ++r) {
        a.in[r] = L.src[r];
        a.out[r] = L.dst[r];
        a.ids[r] = N.ids ? N.ids[r] : nullptr;
        a.valid[r] = N.valid ? N.valid[r] : nullptr;
        vec = vec && uintptr_t(L.src[r]) % 16 == 0 && (!bwd || uintptr_t(L.dst[r]) % 16 == 0);
    }
    a.rows = N.rows;
    a.p = uint32_t(L.p);
    a.experts = N.experts;
    a.k = N.k;
    a.by_k = fast_div(N.k);
    a.by_choices = fast_div(N.rows ? uint32_t(N.rows * N.k) : 1);
    a.by_rows = fast_div(N.rows ? uint32_t(N.rows) : 1);
    a.pass = N.pass;
    a.has_valid = N.valid ? 1 : 0;
    const uint64_t choices = uint64_t(L.p) * N.rows * N.k, cells = uint64_t(L.p) * N.experts;
    a.count_here = fwd && choices <= kCountHereIds && cells <= kCountHereCells;
    a.coef = N.coef;
    a.dloss = N.dloss;
    a.counts = N.counts;
    a.tokens = N.tokens;
    a.loss = N.loss;
    a.ticket = static_cast<unsigned *>(N.scratch);
    a.partials = reinterpret_cast<double2 *>(static_cast<char *>(N.scratch) + kScratchHead);
    a.cells = N.counts;
    a.cell_tokens = N.tokens;
    const bool scratch = fwd && cells <= kScratchCells;
    if (scratch) {
        a.cells = reinterpret_cast<int32_t *>(a.partials + kMaxPartials);
        a.cell_tokens = a.cells + kScratchCells;
    }
    a.cell_room = scratch ? kScratchCells : uint32_t(cells);
    a.status = L.status;
    a.held = N.rows - (L.stall_test == 2 && N.rows ? 1 : 0);
    cudaError_t err = cudaSuccess;
    info->kernels = 0;
    void (*kern)(BalanceArgs<PM>) = balance_any_kernel<T, PM>;
    int lanes = 32, per_sm = 6;      // CTAs that an SM holds at once: the kernels' launch bounds; this one's registers
    size_t smem = size_t(N.experts) * 4 + (a.count_here ? size_t(cells + L.p) * 4 : 0);
    if (!vec && N.experts <= 1024) {
        lanes = 1;
        while (lanes < 32 && uint32_t(lanes) * 16 < N.experts) lanes *= 2;
        switch (lanes) {
        case 1: err = odd_kernel<T, PM, 1, 16>(L.device, &kern); break;
        case 2: err = odd_kernel<T, PM, 2, 16>(L.device, &kern); break;
        case 4: err = odd_kernel<T, PM, 4, 16>(L.device, &kern); break;
        case 8: err = odd_kernel<T, PM, 8, 16>(L.device, &kern); break;
        case 16: err = odd_kernel<T, PM, 16, 16>(L.device, &kern); break;
        default:
            if (N.experts <= 512) err = odd_kernel<T, PM, 32, 16>(L.device, &kern);
            else err = odd_kernel<T, PM, 32, 32>(L.device, &kern);
        }
        if (err != cudaSuccess) return err;
        const bool wide = N.experts > 512;
        per_sm = wide ? kOddCtas<32> : kOddCtas<16>;
        smem += kBalanceWarps * ((wide ? kOddStages<32> : kOddStages<16>) + 1) * size_t(odd_span(32 / lanes, N.experts * (16 / VEC))) + (N.experts * (16 / VEC) + 15) / 16 * 16 + kOddSlack;
    } else if (vec && N.experts <= 1024) {
        per_sm = N.experts > 512 ? 2 : NV > 2 ? 3 : 4;
        lanes = 1;
        while (lanes < 32 && uint32_t(lanes) * 16 < N.experts) lanes *= 2;
        switch (lanes) {
        case 1: kern = balance_kernel<T, PM, 1, NV>; break;
        case 2: kern = balance_kernel<T, PM, 2, NV>; break;
        case 4: kern = balance_kernel<T, PM, 4, NV>; break;
        case 8: kern = balance_kernel<T, PM, 8, NV>; break;
        case 16: kern = balance_kernel<T, PM, 16, NV>; break;
        default:
            if (N.experts <= 512) kern = balance_kernel<T, PM, 32, NV>;
            else kern = balance_kernel<T, PM, 32, 2 * NV>;
        }
    }
    if (fwd && !a.count_here) {
        // the scratch counters are zero already: the call that used them last left them so
        if (!scratch) err = cudaMemsetAsync(N.counts, 0, cells * 4, L.stream);
        if (!scratch && err == cudaSuccess) err = cudaMemsetAsync(N.tokens, 0, size_t(L.p) * 4, L.stream);
        if (err != cudaSuccess) return err;
        // one CTA per SM: every CTA ends with an atomic per expert it met
        const uint64_t want = (N.rows * N.k + kCountThreads - 1) / kCountThreads;
        const uint64_t most = uint64_t(L.num_sms) / uint64_t(L.p) + 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(want < 1 ? 1 : want < most ? want : most), unsigned(L.p));
        cfg.blockDim = dim3(kCountThreads);
        cfg.dynamicSmemBytes = size_t(N.experts) * 4;
        cfg.stream = L.stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        err = cudaLaunchKernelEx(&cfg, balance_count_kernel<PM>, a);
        if (err != cudaSuccess) return err;
        ++info->kernels;
    }
    const uint64_t rows_per_cta = uint64_t(kBalanceWarps) * (32 / lanes);
    const uint64_t want = (N.rows + rows_per_cta - 1) / rows_per_cta;
    const uint64_t all = uint64_t(per_sm) * L.num_sms < kMaxPartials ? uint64_t(per_sm) * L.num_sms : kMaxPartials, most = all / L.p;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(want < 1 ? 1 : want < most ? want : most), unsigned(L.p));
    cfg.blockDim = dim3(kBalanceThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kern, a);
    if (err != cudaSuccess) {
        // what the counting kernel leaves in the scratch is cleared behind it: the next call finds it at zero
        if (scratch && !a.count_here) cudaMemsetAsync(a.cells, 0, size_t(kScratchCells + kMaxRanks) * 4, L.stream);
        return err;
    }
    info->kernel = "balance_loss";
    info->grid = int(cfg.gridDim.x * cfg.gridDim.y);
    info->block = kBalanceThreads;
    info->smem = cfg.dynamicSmemBytes;
    ++info->kernels;
    return cudaGetLastError();
}

template <typename T>
static cudaError_t balance_dtype(const Launch &L, const BalanceLaunch &N, LaunchInfo *info)
{
    return L.p <= 8 ? balance_shape<T, 8>(L, N, info) : balance_shape<T, kMaxRanks>(L, N, info);
}

cudaError_t launch_balance(const Launch &L, const BalanceLaunch &N, LaunchInfo *info)
{
    switch (L.dtype) {
    case DT_F32: return balance_dtype<F32>(L, N, info);
    case DT_F16: return balance_dtype<F16>(L, N, info);
    case DT_BF16: return balance_dtype<BF16>(L, N, info);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace ccl
