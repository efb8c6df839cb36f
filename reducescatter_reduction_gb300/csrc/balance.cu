// The load-balance loss of a router over p data-parallel ranks: per-expert
// counts, the loss, and the gradient of the router's logits.
//
// With N the valid rows of all ranks, count_e the valid rows' choices of
// expert e over all ranks and p_t the softmax of row t:
//   loss = coef E sum_e f_e P_e,  f_e = count_e / (k N),  P_e = (1/N) sum_t p_te
//   dx_te = dloss p_te (a_e - sum_j p_tj a_j),  a_e = coef E count_e / (k N^2)
// Both need the counts only as a_e, so once the choices are counted one pass
// over the logits gives loss = sum_t sum_e p_te a_e and the gradient together.
// Differences of nearly equal a_e make the gradient: they are formed from the
// integer counts in fp64 as d_e = a_e - mean(a) before fp32 sees them;
// p_te (d_e - sum_j p_tj d_j) is the same gradient, and the loss is
// mean(a) (rows with a softmax) + sum_t sum_e p_te d_e.
#include "logits.cuh"

namespace ccl {

constexpr int kBalanceThreads = 256;
constexpr int kBalanceWarps = kBalanceThreads / 32;
// Up to this many choices and counters in all, every CTA counts for itself
// instead of waiting for a counting kernel.
constexpr uint64_t kCountHereIds = 8192;
constexpr uint64_t kCountHereCells = 4096;

template <int PM>
struct BalanceArgs {
    const void *in[PM];
    void *out[PM];
    const int32_t *ids[PM];
    const uint8_t *valid[PM];
    uint64_t rows;
    uint32_t p, experts, k;
    FastDiv by_k;
    int pass, has_valid, count_here;
    double coef;
    const float *dloss;
    int32_t *counts, *tokens;
    float *loss;
    unsigned *ticket;
    double2 *partials;
    unsigned *status;
};

// Adds rank r's choices [j0, j1) with the given stride to hist[experts].
template <int PM>
__device__ __forceinline__ void count_choices(const BalanceArgs<PM> &a, uint32_t r, uint32_t first, uint32_t stride, int *hist)
{
    const uint32_t n = uint32_t(a.rows) * a.k;
    for (uint64_t j = first; j < n; j += stride) {
        const int id = a.ids[r][j];
        if (uint32_t(id) >= a.experts) continue;
        if (a.has_valid && !a.valid[r][div_by(uint32_t(j), a.by_k)]) continue;
        atomicAdd(&hist[id], 1);
    }
}

template <int PM>
__device__ __forceinline__ int count_rows(const BalanceArgs<PM> &a, uint32_t r, uint32_t first, uint32_t stride)
{
    int n = 0;
    for (uint64_t t = first; t < a.rows; t += stride) n += a.valid[r][t] != 0;
    return n;
}

// Counts the choices of all ranks into counts and tokens, which are zero.
template <int PM>
__global__ void __launch_bounds__(kBalanceThreads) balance_count_kernel(const __grid_constant__ BalanceArgs<PM> a)
{
    extern __shared__ int hist[];
    const uint32_t r = blockIdx.y;
    for (uint32_t e = threadIdx.x; e < a.experts; e += kBalanceThreads) hist[e] = 0;
    grid_dependency_wait();
    grid_dependents_launch();
    __syncthreads();
    const uint32_t first = blockIdx.x * kBalanceThreads + threadIdx.x, stride = gridDim.x * kBalanceThreads;
    count_choices(a, r, first, stride, hist);
    if (a.has_valid) {
        int n = count_rows(a, r, first, stride);
        n = __reduce_add_sync(0xffffffffu, n);
        if (threadIdx.x % 32 == 0 && n) atomicAdd(&a.tokens[r], n);
    } else if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.tokens[r] = int(a.rows);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.experts; e += kBalanceThreads)
        if (hist[e]) atomicAdd(&a.counts[uint64_t(r) * a.experts + e], hist[e]);
}

// d_e into shared memory; returns mean(a).  hist: p * experts counters and p
// row counts when the CTA counts for itself.
template <int PM>
__device__ __forceinline__ float balance_coefficients(const BalanceArgs<PM> &a, float *d_s, int *hist)
{
    __shared__ unsigned long long sums[2];
    const uint32_t E = a.experts;
    if (threadIdx.x < 2) sums[threadIdx.x] = 0;
    const int32_t *counts = a.counts, *tokens = a.tokens;
    if (a.count_here) {
        int *rows_s = hist + a.p * E;
        for (uint32_t i = threadIdx.x; i < a.p * E + a.p; i += kBalanceThreads) hist[i] = 0;
        grid_dependency_wait();
        __syncthreads();
        for (uint32_t r = 0; r < a.p; ++r) {
            count_choices(a, r, threadIdx.x, kBalanceThreads, hist + r * E);
            int n = a.has_valid ? count_rows(a, r, threadIdx.x, kBalanceThreads) : threadIdx.x == 0 ? int(a.rows) : 0;
            n = __reduce_add_sync(0xffffffffu, n);
            if (threadIdx.x % 32 == 0 && n) atomicAdd(&rows_s[r], n);
        }
        __syncthreads();
        if (blockIdx.x == 0 && blockIdx.y == 0) {
            for (uint32_t i = threadIdx.x; i < a.p * E; i += kBalanceThreads) a.counts[i] = hist[i];
            for (uint32_t r = threadIdx.x; r < a.p; r += kBalanceThreads) a.tokens[r] = rows_s[r];
        }
        counts = hist;
        tokens = rows_s;
    } else {
        grid_dependency_wait();
        __syncthreads();
    }
    // sums of integers: any order gives the same
    for (uint32_t r = threadIdx.x; r < a.p; r += kBalanceThreads) atomicAdd(&sums[0], (unsigned long long)tokens[r]);
    unsigned long long mine = 0;
    for (uint32_t e = threadIdx.x; e < E; e += kBalanceThreads) {
        for (uint32_t r = 0; r < a.p; ++r) mine += (unsigned long long)(long long)counts[uint64_t(r) * E + e];
    }
    if (mine) atomicAdd(&sums[1], mine);
    __syncthreads();
    const double n = double(sums[0]), mean = double(sums[1]) / double(E);
    const double scale = sums[0] ? a.coef * double(E) / (double(a.k) * n * n) : 0.0;
    for (uint32_t e = threadIdx.x; e < E; e += kBalanceThreads) {
        long long total = 0;
        for (uint32_t r = 0; r < a.p; ++r) total += counts[uint64_t(r) * E + e];
        d_s[e] = float((double(total) - mean) * scale);
    }
    __syncthreads();
    return float(mean * scale);
}

// The CTAs' sums: each leaves its pair, the last one adds the pairs in the
// order of the CTAs, writes the loss and leaves the ticket at zero.
template <int PM>
__device__ __forceinline__ void balance_finish(const BalanceArgs<PM> &a, float lean, int live, float mean)
{
    __shared__ double red[2][kBalanceWarps];
    __shared__ bool last;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    double s = lean, c = live;
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
    const unsigned grid = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
    if (threadIdx.x == 0) {
        s = c = 0.0;
        for (int w = 0; w < kBalanceWarps; ++w) {
            s += red[0][w];
            c += red[1][w];
        }
        a.partials[me] = make_double2(s, c);
        __threadfence();
        last = atomicAdd(a.ticket, 1u) == grid - 1;
    }
    __syncthreads();
    if (!last || warp != 0) return;
    __threadfence();
    s = c = 0.0;
    for (unsigned i = lane; i < grid; i += 32) {
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
        *a.loss = float(s + c * double(mean));
        *a.ticket = 0;
    }
}

// L lanes of a warp take a row, 16-byte groups l, l + L, ... of it; NV groups
// a lane hold the whole row, so the logits are read once.
template <typename T, int PM, int L, int NV>
__global__ void __launch_bounds__(kBalanceThreads) balance_kernel(const __grid_constant__ BalanceArgs<PM> a)
{
    using Tr = Traits<T>;
    constexpr int VEC = Tr::VEC, S = 16 / VEC, RPW = 32 / L;
    extern __shared__ float d_s[];
    const uint32_t E = a.experts, r = blockIdx.y;
    const float mean = balance_coefficients(a, d_s, reinterpret_cast<int *>(d_s + E));
    grid_dependents_launch();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, l = lane % L;
    float d[NV * VEC];
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const uint32_t col = (n * L + l) * VEC + i;
            d[n * VEC + i] = col < E ? d_s[col] : 0.0f;
        }
    const uint32_t low = VEC == 4 ? 0xff800000u : Tr::kDtype == DT_BF16 ? 0xff80ff80u : 0xfc00fc00u;   // -inf
    const bool fwd = a.pass & CCL_PASS_FORWARD, bwd = a.pass & CCL_PASS_BACKWARD;
    const float up = bwd && a.dloss ? *a.dloss : 1.0f;
    const char *in = static_cast<const char *>(a.in[r]);
    char *out = static_cast<char *>(a.out[r]);
    const uint64_t stride = uint64_t(gridDim.x) * kBalanceWarps * RPW;
    auto fetch = [&](uint64_t t, uint4 (&raw)[NV]) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const uint32_t col = (n * L + l) * VEC;
            raw[n] = t < a.rows && col < E && in_bounds(col + VEC <= E, a.status, kSiteBalance, t)
                         ? ld_coherent_v4(in + (t * E + col) * S)
                         : make_uint4(low, low, low, low);
        }
    };
    float lean_sum = 0.0f;
    int live = 0;
    uint64_t base = (uint64_t(blockIdx.x) * kBalanceWarps + warp) * RPW;
    uint4 raw[NV];
    fetch(base + lane / L, raw);
    for (; base < a.rows; base += stride) {
        const uint64_t t = base + lane / L;
        const bool valid = t < a.rows && (!a.has_valid || a.valid[r][t]);
        float x[NV * VEC], m = -INFINITY;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float f[VEC];
            Tr::unpack(raw[n], f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[n * VEC + i] = f[i];
        }
        fetch(t + stride, raw);
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) m = fmaxf(m, x[i]);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = m == -INFINITY ? 0.0f : m;
        float s = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) {
            x[i] = ex2((x[i] - m) * kLog2e);
            s += x[i];
            dot = fmaf(x[i], d[i], dot);
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        const float inv = s == 0.0f ? 0.0f : 1.0f / s;    // a row of nothing but -inf has no softmax: p = 0
        const float lean = dot * inv;
        if (valid && l == 0 && s != 0.0f) {
            lean_sum += lean;
            ++live;
        }
        if (bwd && t < a.rows) {
            const float g = inv * up;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const uint32_t col = (n * L + l) * VEC;
                if (col >= E) continue;
                float f[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[i] = valid ? x[n * VEC + i] * (d[n * VEC + i] - lean) * g : 0.0f;
                if (in_bounds(col + VEC <= E, a.status, kSiteBalance, t)) st_stream_v4(out + (t * E + col) * S, Tr::pack(f));
            }
        }
    }
    if (fwd) balance_finish(a, lean_sum, live, mean);
}

// Any number of experts and any alignment: a warp per row, element by
// element, the row read once per step (the later reads from cache).
template <typename T, int PM>
__global__ void __launch_bounds__(kBalanceThreads) balance_any_kernel(const __grid_constant__ BalanceArgs<PM> a)
{
    using Tr = Traits<T>;
    extern __shared__ float d_s[];
    const uint32_t E = a.experts, r = blockIdx.y;
    const float mean = balance_coefficients(a, d_s, reinterpret_cast<int *>(d_s + E));
    grid_dependents_launch();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const bool fwd = a.pass & CCL_PASS_FORWARD, bwd = a.pass & CCL_PASS_BACKWARD;
    const float up = bwd && a.dloss ? *a.dloss : 1.0f;
    float lean_sum = 0.0f;
    int live = 0;
    for (uint64_t t = uint64_t(blockIdx.x) * kBalanceWarps + warp; t < a.rows; t += uint64_t(gridDim.x) * kBalanceWarps) {
        const uint64_t at = t * E;
        const bool valid = !a.has_valid || a.valid[r][t];
        if (!valid) {
            if (bwd)
                for (uint32_t e = lane; e < E; e += 32)
                    if (in_bounds(t < a.rows, a.status, kSiteBalance, t)) Tr::store1(a.out[r], at + e, 0.0f);
            continue;
        }
        float m = -INFINITY;
        for (uint32_t e = lane; e < E; e += 32)
            if (in_bounds(t < a.rows, a.status, kSiteBalance, t)) m = fmaxf(m, Tr::load1(a.in[r], at + e));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = m == -INFINITY ? 0.0f : m;
        float s = 0.0f, dot = 0.0f;
        for (uint32_t e = lane; e < E; e += 32) {
            const float v = ex2((Tr::load1(a.in[r], at + e) - m) * kLog2e);
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
                const float v = ex2((Tr::load1(a.in[r], at + e) - m) * kLog2e);
                Tr::store1(a.out[r], at + e, v * (d_s[e] - lean) * g);
            }
        }
    }
    if (fwd) balance_finish(a, lean_sum, live, mean);
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
    a.status = L.status;
    cudaError_t err = cudaSuccess;
    info->kernels = 0;
    if (fwd && !a.count_here) {
        err = cudaMemsetAsync(N.counts, 0, cells * 4, L.stream);
        if (err == cudaSuccess) err = cudaMemsetAsync(N.tokens, 0, size_t(L.p) * 4, L.stream);
        if (err != cudaSuccess) return err;
        const uint64_t want = (N.rows * N.k + 4 * kBalanceThreads - 1) / (4 * kBalanceThreads);
        const uint64_t most = uint64_t(4 * L.num_sms) / uint64_t(L.p) + 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(want < 1 ? 1 : want < most ? want : most), unsigned(L.p));
        cfg.blockDim = dim3(kBalanceThreads);
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
    void (*kern)(BalanceArgs<PM>) = balance_any_kernel<T, PM>;
    int lanes = 32;
    if (vec && N.experts <= 1024) {
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
    const uint64_t rows_per_cta = uint64_t(kBalanceWarps) * (32 / lanes);
    const uint64_t want = (N.rows + rows_per_cta - 1) / rows_per_cta;
    const uint64_t most = uint64_t(6 * L.num_sms) < kMaxPartials ? uint64_t(6 * L.num_sms) / L.p : kMaxPartials / L.p;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(want < 1 ? 1 : want < most ? want : most), unsigned(L.p));
    cfg.blockDim = dim3(kBalanceThreads);
    cfg.dynamicSmemBytes = size_t(N.experts) * 4 + (a.count_here ? size_t(cells + L.p) * 4 : 0);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kern, a);
    if (err != cudaSuccess) return err;
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
