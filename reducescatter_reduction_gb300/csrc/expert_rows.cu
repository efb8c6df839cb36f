// Tokens to the rows of their experts and back: dispatch, combine and
// combine's gradient over p ranks' buffers.
//
//   dispatch  row[slot_tj] = w_tj x_t
//   combine   y_t          = sum_j w_tj row[slot_tj]
//   gradient  drow[slot_tj] = w_tj dy_t,  dw_tj = <dy_t, row[slot_tj]>
// Each is driven by the tokens: a CTA takes one, so a token's row is read (or
// written) once and its k expert rows once each, which is all the traffic there has to be.
#include "logits.cuh"

namespace ccl {

constexpr unsigned kSiteExperts = 11;
constexpr int kRowsThreads = 256;

template <int PM>
struct RowsArgs {
    const void *in[PM];
    void *out[PM];
    const int32_t *slots[PM];
    const float *weights[PM];
    const void *experts[PM];
    float *dweights[PM];
    uint64_t hidden;
    uint32_t rows, p, k, capacity, slot_end;   // slot_end: p * capacity
    FastDiv by_rows, by_capacity;
    int weighted;
    // checked build:
    unsigned *status;
    uint32_t held;        // tokens that every token buffer and list has: `rows`, or one less where the debug hook wants the checks to fail
};

template <int PM>
__device__ __forceinline__ bool token_held(const RowsArgs<PM> &a, const void *buf, const void *at, uint32_t bytes, uint32_t element)
{
    return !kBoundsCheck || in_buffer(at, bytes, buf, uint64_t(a.held) * a.hidden * element, a.status, kSiteExperts);
}
template <int PM>
__device__ __forceinline__ bool row_of_expert_held(const RowsArgs<PM> &a, const void *buf, const void *at, uint32_t bytes, uint32_t element)
{
    return !kBoundsCheck || in_buffer(at, bytes, buf, uint64_t(a.capacity) * a.hidden * element, a.status, kSiteExperts);
}
template <int PM>
__device__ __forceinline__ bool entry_held(const RowsArgs<PM> &a, uint64_t entry)
{
    return in_bounds(entry < uint64_t(a.held) * a.k, a.status, kSiteExperts, entry);
}

// A unit of a row: a 16-byte group, or one element where rows are not groups.
template <typename T, bool VECTOR>
struct RowUnit;
template <typename T>
struct RowUnit<T, true> {
    using Tr = Traits<T>;
    static constexpr int N = Tr::VEC, BYTES = 16;
    using Raw = uint4;
    __device__ static __forceinline__ Raw load(const void *p) { return ld_stream_v4(p); }
    __device__ static __forceinline__ void store(void *p, const Raw &v) { st_stream_v4(p, v); }
    __device__ static __forceinline__ void unpack(const Raw &v, typename Tr::Acc (&f)[N]) { Tr::unpack(v, f); }
    __device__ static __forceinline__ Raw pack(const typename Tr::Acc (&f)[N]) { return Tr::pack(f); }
};
template <typename T>
struct RowUnit<T, false> {
    using Tr = Traits<T>;
    static constexpr int N = 1, BYTES = 16 / Tr::VEC;
    using Raw = typename std::conditional<BYTES == 2, uint16_t, uint32_t>::type;
    __device__ static __forceinline__ Raw load(const void *p) { return *static_cast<const Raw *>(p); }
    __device__ static __forceinline__ void store(void *p, const Raw &v) { *static_cast<Raw *>(p) = v; }
    __device__ static __forceinline__ void unpack(const Raw &v, typename Tr::Acc (&f)[1]) { f[0] = Tr::load1(&v, 0); }
    __device__ static __forceinline__ Raw pack(const typename Tr::Acc (&f)[1])
    {
        Raw v;
        Tr::store1(&v, 0, f[0]);
        return v;
    }
};

// One choice of the CTA's token: where its row begins, and its weight.
struct Choice {
    char *row;            // null: none
    float weight;
    uint32_t rank;
};

// Choices first, first + 1, ... of token `t` of rank `r` into shared memory; `of` has the experts' buffers.
template <int PM>
__device__ __forceinline__ void read_choices(const RowsArgs<PM> &a, uint32_t r, uint32_t t, const void *const *of, uint32_t element,
                                             Choice *list)
{
    for (uint32_t j = threadIdx.x; j < a.k; j += kRowsThreads) {
        const uint64_t entry = uint64_t(t) * a.k + j;
        Choice c = {nullptr, 1.0f, 0};
        if (entry_held(a, entry)) {
            const uint32_t slot = uint32_t(a.slots[r][entry]);
            if (a.weighted) c.weight = a.weights[r][entry];
            if (slot < a.slot_end) {
                c.rank = div_by(slot, a.by_capacity);
                c.row = static_cast<char *>(const_cast<void *>(of[c.rank])) + uint64_t(slot - c.rank * a.capacity) * a.hidden * element;
            }
        }
        list[j] = c;
    }
    __syncthreads();
}

template <typename T, int PM, bool VECTOR>
__global__ void __launch_bounds__(kRowsThreads) dispatch_kernel(const __grid_constant__ RowsArgs<PM> a)
{
    using U = RowUnit<T, VECTOR>;
    constexpr uint32_t S = 16 / Traits<T>::VEC;
    extern __shared__ Choice list[];
    grid_dependency_wait();
    grid_dependents_launch();
    const uint32_t r = div_by(blockIdx.x, a.by_rows), t = blockIdx.x - r * a.rows;
    read_choices(a, r, t, a.out, S, list);
    const char *token = static_cast<const char *>(a.in[r]) + uint64_t(t) * a.hidden * S;
    const uint64_t units = a.hidden / U::N;
    for (uint64_t u = threadIdx.x; u < units; u += kRowsThreads) {
        if (!token_held(a, a.in[r], token + u * U::BYTES, U::BYTES, S)) continue;
        const typename U::Raw v = U::load(token + u * U::BYTES);
        typename Traits<T>::Acc f[U::N], g[U::N];
        U::unpack(v, f);
        for (uint32_t j = 0; j < a.k; ++j) {
            const Choice c = list[j];
            if (!c.row || !row_of_expert_held(a, a.out[c.rank], c.row + u * U::BYTES, U::BYTES, S)) continue;
            typename U::Raw w = v;
            if constexpr (!std::is_same<T, I32>::value) {
                if (a.weighted) {
#pragma unroll
                    for (int i = 0; i < U::N; ++i) g[i] = __fmul_rn(f[i], c.weight);
                    w = U::pack(g);
                }
            }
            U::store(c.row + u * U::BYTES, w);
        }
    }
}

template <typename T, int PM, bool VECTOR>
__global__ void __launch_bounds__(kRowsThreads) combine_kernel(const __grid_constant__ RowsArgs<PM> a)
{
    using U = RowUnit<T, VECTOR>;
    constexpr uint32_t S = 16 / Traits<T>::VEC;
    extern __shared__ Choice list[];
    grid_dependency_wait();
    grid_dependents_launch();
    const uint32_t r = div_by(blockIdx.x, a.by_rows), t = blockIdx.x - r * a.rows;
    read_choices(a, r, t, a.in, S, list);
    char *token = static_cast<char *>(a.out[r]) + uint64_t(t) * a.hidden * S;
    const uint64_t units = a.hidden / U::N;
    for (uint64_t u = threadIdx.x; u < units; u += kRowsThreads) {
        float sum[U::N], f[U::N];
#pragma unroll
        for (int i = 0; i < U::N; ++i) sum[i] = 0.0f;
        for (uint32_t j = 0; j < a.k; ++j) {
            const Choice c = list[j];
            if (!c.row || !row_of_expert_held(a, a.in[c.rank], c.row + u * U::BYTES, U::BYTES, S)) continue;
            U::unpack(U::load(c.row + u * U::BYTES), f);
#pragma unroll
            for (int i = 0; i < U::N; ++i) sum[i] = fmaf(c.weight, f[i], sum[i]);
        }
        if (token_held(a, a.out[r], token + u * U::BYTES, U::BYTES, S)) U::store(token + u * U::BYTES, U::pack(sum));
    }
}

template <typename T, int PM, bool VECTOR>
__global__ void __launch_bounds__(kRowsThreads) combine_grad_kernel(const __grid_constant__ RowsArgs<PM> a)
{
    using U = RowUnit<T, VECTOR>;
    constexpr uint32_t S = 16 / Traits<T>::VEC;
    constexpr int KB = 8;      // choices whose products are summed at a time
    extern __shared__ Choice list[];
    __shared__ float parts[kRowsThreads / 32][KB];
    grid_dependency_wait();
    grid_dependents_launch();
    const uint32_t r = div_by(blockIdx.x, a.by_rows), t = blockIdx.x - r * a.rows;
    read_choices(a, r, t, a.out, S, list);
    const char *token = static_cast<const char *>(a.in[r]) + uint64_t(t) * a.hidden * S;
    const uint64_t units = a.hidden / U::N;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (uint32_t first = 0; first < a.k; first += KB) {
        float sum[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) sum[j] = 0.0f;
        for (uint64_t u = threadIdx.x; u < units; u += kRowsThreads) {
            if (!token_held(a, a.in[r], token + u * U::BYTES, U::BYTES, S)) continue;
            float f[U::N], g[U::N];
            U::unpack(U::load(token + u * U::BYTES), f);
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                if (first + j >= a.k) break;
                const Choice c = list[first + j];
                if (!c.row || !row_of_expert_held(a, a.out[c.rank], c.row + u * U::BYTES, U::BYTES, S)) continue;
                const char *z = static_cast<const char *>(a.experts[c.rank]) + (c.row - static_cast<char *>(a.out[c.rank]));
                U::unpack(U::load(z + u * U::BYTES), g);
#pragma unroll
                for (int i = 0; i < U::N; ++i) sum[j] = fmaf(f[i], g[i], sum[j]);
#pragma unroll
                for (int i = 0; i < U::N; ++i) g[i] = __fmul_rn(f[i], c.weight);
                U::store(c.row + u * U::BYTES, U::pack(g));
            }
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
            if (lane == 0) parts[warp][j] = sum[j];
        }
        __syncthreads();
        if (threadIdx.x < KB && first + threadIdx.x < a.k) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kRowsThreads / 32; ++w) s += parts[w][threadIdx.x];
            const uint64_t entry = uint64_t(t) * a.k + first + threadIdx.x;
            if (entry_held(a, entry)) a.dweights[r][entry] = s;
        }
        __syncthreads();
    }
}

template <typename T, int PM, bool VECTOR>
static cudaError_t rows_launch(const Launch &L, const RowsLaunch &N, LaunchInfo *info)
{
    RowsArgs<PM> a = {};
    for (int r = 0; r < L.p; ++r) {
        a.in[r] = L.src[r];
        a.out[r] = L.dst[r];
        a.slots[r] = N.slots[r];
        a.weights[r] = N.weights ? N.weights[r] : nullptr;
        a.experts[r] = N.experts ? N.experts[r] : nullptr;
        a.dweights[r] = N.dweights ? N.dweights[r] : nullptr;
    }
    a.hidden = N.hidden;
    a.rows = uint32_t(N.rows);
    a.p = uint32_t(L.p);
    a.k = N.k;
    a.capacity = N.capacity;
    a.slot_end = N.capacity * uint32_t(L.p);
    a.by_rows = fast_div(a.rows);
    a.by_capacity = fast_div(N.capacity ? N.capacity : 1);
    a.weighted = N.weights ? 1 : 0;
    a.status = L.status;
    a.held = a.rows - (L.stall_test == 2 ? 1 : 0);
    const unsigned grid = a.rows * a.p;
    const size_t smem = N.k * sizeof(Choice);
    static std::atomic<unsigned long long> ready[3];
    void (*kern)(RowsArgs<PM>) = nullptr;
    if constexpr (std::is_same<T, I32>::value)
        kern = dispatch_kernel<T, PM, VECTOR>;
    else
        kern = N.op == ROWS_DISPATCH ? dispatch_kernel<T, PM, VECTOR> : N.op == ROWS_COMBINE ? combine_kernel<T, PM, VECTOR> : combine_grad_kernel<T, PM, VECTOR>;
    cudaError_t err = smem > 48 * 1024 ? allow_dynamic_smem(kern, 4096 * sizeof(Choice), L.device, ready[N.op]) : cudaSuccess;
    if (err == cudaSuccess) err = launch_dependent(kern, grid, kRowsThreads, smem, L.stream, a);
    if (err != cudaSuccess) return err;
    info->kernel = N.op == ROWS_DISPATCH ? "expert_dispatch" : N.op == ROWS_COMBINE ? "expert_combine" : "expert_combine_grad";
    info->grid = int(grid);
    info->block = kRowsThreads;
    info->smem = smem;
    info->kernels = 1;
    return cudaSuccess;
}

template <typename T>
static cudaError_t rows_dtype(const Launch &L, const RowsLaunch &N, LaunchInfo *info)
{
    if (L.p <= 8) return L.vec ? rows_launch<T, 8, true>(L, N, info) : rows_launch<T, 8, false>(L, N, info);
    return L.vec ? rows_launch<T, kMaxRanks, true>(L, N, info) : rows_launch<T, kMaxRanks, false>(L, N, info);
}

cudaError_t launch_expert_rows(const Launch &L, const RowsLaunch &N, LaunchInfo *info)
{
    switch (L.dtype) {
    case DT_F32: return rows_dtype<F32>(L, N, info);
    case DT_F16: return rows_dtype<F16>(L, N, info);
    case DT_BF16: return rows_dtype<BF16>(L, N, info);
    default: return rows_dtype<I32>(L, N, info);
    }
}

}  // namespace ccl
