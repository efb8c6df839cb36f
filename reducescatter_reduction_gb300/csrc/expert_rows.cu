// Tokens to the rows of their experts and back: dispatch, combine and
// combine's gradient over p ranks' buffers.
//
//   dispatch  row[slot_tj] = w_tj x_t
//   combine   y_t          = sum_j w_tj row[slot_tj]
//   gradient  drow[slot_tj] = w_tj dy_t,  dw_tj = <dy_t, row[slot_tj]>
// Each is driven by the tokens: a team of 32 to 256 threads takes one, so a
// token's row is read (or written) once and its k expert rows once each, which
// is all the traffic there has to be.  A thread loads a batch of KB choices of
// UN units before it uses the first.
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
    int team_shift;       // a team has 2^team_shift threads
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

// A unit of a row: 16 bytes, 4 bytes or one element.
template <typename T, int BYTES>
struct RowUnit {
    using Tr = Traits<T>;
    using Acc = typename Tr::Acc;
    static constexpr int S = 16 / Tr::VEC, N = BYTES / S;
    using Raw = typename std::conditional<BYTES == 16, uint4, typename std::conditional<BYTES == 4, uint32_t, uint16_t>::type>::type;
    __device__ static __forceinline__ Raw zero()
    {
        if constexpr (BYTES == 16) return make_uint4(0, 0, 0, 0);
        else return Raw(0);
    }
    __device__ static __forceinline__ Raw load(const void *p)
    {
        if constexpr (BYTES == 16) return ld_stream_v4(p);
        else return __ldg(static_cast<const Raw *>(p));
    }
    __device__ static __forceinline__ void store(void *p, const Raw &v)
    {
        if constexpr (BYTES == 16) st_stream_v4(p, v);
        else *static_cast<Raw *>(p) = v;
    }
    __device__ static __forceinline__ void unpack(const Raw &v, Acc (&f)[N])
    {
        if constexpr (BYTES == 16) {
            Tr::unpack(v, f);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = Tr::load1(&v, i);
        }
    }
    __device__ static __forceinline__ Raw pack(const Acc (&f)[N])
    {
        if constexpr (BYTES == 16) {
            return Tr::pack(f);
        } else {
            Raw v;
#pragma unroll
            for (int i = 0; i < N; ++i) Tr::store1(&v, i, f[i]);
            return v;
        }
    }
};

// One choice of a team's token: where its row begins, and its weight.
struct Choice {
    char *row;            // null: none
    float weight;
    uint32_t rank;
};

// A team of threads, its token and its choices.
template <int PM>
struct Team {
    uint32_t thread, threads;   // of the team
    uint32_t rank, token;
    uint64_t first, end;        // the team's units
    bool on;                    // it has a token
    Choice *list;

    // `of` has the experts' buffers; `list` room for the choices of all teams.
    __device__ __forceinline__ Team(const RowsArgs<PM> &a, const void *const *of, uint32_t S, uint32_t bytes, Choice *all)
    {
        threads = 1u << a.team_shift;
        thread = threadIdx.x & (threads - 1);
        const uint32_t team = threadIdx.x >> a.team_shift, t = blockIdx.x * (kRowsThreads >> a.team_shift) + team;
        on = t < a.rows * a.p;
        rank = on ? div_by(t, a.by_rows) : 0;
        token = t - rank * a.rows;
        const uint64_t units = a.hidden * S / bytes;
        first = units * blockIdx.y / gridDim.y + thread;
        end = on ? units * (blockIdx.y + 1) / gridDim.y : 0;
        list = all + team * a.k;
        for (uint32_t j = thread; j < a.k; j += threads) {
            const uint64_t entry = uint64_t(token) * a.k + j;
            Choice c = {nullptr, 1.0f, 0};
            if (on && entry_held(a, entry)) {
                const uint32_t slot = uint32_t(a.slots[rank][entry]);
                if (a.weighted) c.weight = a.weights[rank][entry];
                if (slot < a.slot_end) {
                    c.rank = div_by(slot, a.by_capacity);
                    c.row = static_cast<char *>(const_cast<void *>(of[c.rank])) + uint64_t(slot - c.rank * a.capacity) * a.hidden * S;
                }
            }
            list[j] = c;
        }
        __syncthreads();
    }
};

template <typename T, int PM, int BYTES, int UN>
__global__ void __launch_bounds__(kRowsThreads) dispatch_kernel(const __grid_constant__ RowsArgs<PM> a)
{
    using U = RowUnit<T, BYTES>;
    constexpr uint32_t S = U::S;
    extern __shared__ Choice lists[];
    grid_dependency_wait();
    grid_dependents_launch();
    const Team<PM> t(a, a.out, S, BYTES, lists);
    const char *token = static_cast<const char *>(a.in[t.rank]) + uint64_t(t.token) * a.hidden * S;
    for (uint64_t u = t.first; u < t.end; u += UN * t.threads) {
        typename U::Raw v[UN];
#pragma unroll
        for (int n = 0; n < UN; ++n) {
            const char *at = token + (u + n * t.threads) * BYTES;
            if (u + n * t.threads < t.end && token_held(a, a.in[t.rank], at, BYTES, S)) v[n] = U::load(at);
        }
        for (uint32_t j = 0; j < a.k; ++j) {
            const Choice c = t.list[j];
            if (!c.row) continue;
#pragma unroll
            for (int n = 0; n < UN; ++n) {
                const uint64_t at = (u + n * t.threads) * BYTES;
                if (u + n * t.threads >= t.end || !token_held(a, a.in[t.rank], token + at, BYTES, S) ||
                    !row_of_expert_held(a, a.out[c.rank], c.row + at, BYTES, S))
                    continue;
                typename U::Raw w = v[n];
                if constexpr (!std::is_same<T, I32>::value) {
                    if (a.weighted) {
                        float f[U::N];
                        U::unpack(w, f);
#pragma unroll
                        for (int i = 0; i < U::N; ++i) f[i] = __fmul_rn(f[i], c.weight);
                        w = U::pack(f);
                    }
                }
                U::store(c.row + at, w);
            }
        }
    }
}

template <typename T, int PM, int BYTES, int KB, int UN>
__global__ void __launch_bounds__(kRowsThreads, BYTES == 16 && KB * UN == 8 ? 3 : 4) combine_kernel(const __grid_constant__ RowsArgs<PM> a)
{
    using U = RowUnit<T, BYTES>;
    constexpr uint32_t S = U::S;
    extern __shared__ Choice lists[];
    grid_dependency_wait();
    grid_dependents_launch();
    const Team<PM> t(a, a.in, S, BYTES, lists);
    char *token = static_cast<char *>(a.out[t.rank]) + uint64_t(t.token) * a.hidden * S;
    for (uint64_t u = t.first; u < t.end; u += UN * t.threads) {
        float sum[UN][U::N];
#pragma unroll
        for (int n = 0; n < UN; ++n)
#pragma unroll
            for (int i = 0; i < U::N; ++i) sum[n][i] = 0.0f;
        for (uint32_t first = 0; first < a.k; first += KB) {
            typename U::Raw z[KB][UN];
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const Choice c = first + j < a.k ? t.list[first + j] : Choice{nullptr, 0.0f, 0};
#pragma unroll
                for (int n = 0; n < UN; ++n) {
                    const char *at = c.row + (u + n * t.threads) * BYTES;
                    z[j][n] = U::zero();
                    if (c.row && u + n * t.threads < t.end && row_of_expert_held(a, a.in[c.rank], at, BYTES, S)) z[j][n] = U::load(at);
                }
            }
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                if (first + j >= a.k) break;
                const Choice c = t.list[first + j];
                if (!c.row) continue;
#pragma unroll
                for (int n = 0; n < UN; ++n) {
                    float f[U::N];
                    U::unpack(z[j][n], f);
#pragma unroll
                    for (int i = 0; i < U::N; ++i) sum[n][i] = fmaf(c.weight, f[i], sum[n][i]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < UN; ++n) {
            char *at = token + (u + n * t.threads) * BYTES;
            if (u + n * t.threads < t.end && token_held(a, a.out[t.rank], at, BYTES, S)) U::store(at, U::pack(sum[n]));
        }
    }
}

template <typename T, int PM, int BYTES, int KB, int UN>
__global__ void __launch_bounds__(kRowsThreads, BYTES == 16 && KB * UN == 8 ? 3 : 4) combine_grad_kernel(const __grid_constant__ RowsArgs<PM> a)
{
    using U = RowUnit<T, BYTES>;
    constexpr uint32_t S = U::S;
    extern __shared__ Choice lists[];
    __shared__ float parts[kRowsThreads / 32][KB];
    grid_dependency_wait();
    grid_dependents_launch();
    const Team<PM> t(a, a.out, S, BYTES, lists);
    const char *token = static_cast<const char *>(a.in[t.rank]) + uint64_t(t.token) * a.hidden * S;
    const uint32_t warps = t.threads / 32, warp = threadIdx.x / 32;
    for (uint32_t first = 0; first < a.k; first += KB) {
        float sum[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) sum[j] = 0.0f;
        for (uint64_t u = t.first; u < t.end; u += UN * t.threads) {
            typename U::Raw v[UN], z[KB][UN];
#pragma unroll
            for (int n = 0; n < UN; ++n) {
                const char *at = token + (u + n * t.threads) * BYTES;
                v[n] = U::zero();
                if (u + n * t.threads < t.end && token_held(a, a.in[t.rank], at, BYTES, S)) v[n] = U::load(at);
            }
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const Choice c = first + j < a.k ? t.list[first + j] : Choice{nullptr, 0.0f, 0};
                const char *row = c.row ? static_cast<const char *>(a.experts[c.rank]) + (c.row - static_cast<char *>(a.out[c.rank])) : nullptr;
#pragma unroll
                for (int n = 0; n < UN; ++n) {
                    const char *at = row + (u + n * t.threads) * BYTES;
                    z[j][n] = U::zero();
                    if (c.row && u + n * t.threads < t.end && row_of_expert_held(a, a.experts[c.rank], at, BYTES, S)) z[j][n] = U::load(at);
                }
            }
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                if (first + j >= a.k) break;
                const Choice c = t.list[first + j];
                if (!c.row) continue;
#pragma unroll
                for (int n = 0; n < UN; ++n) {
                    char *at = c.row + (u + n * t.threads) * BYTES;
                    float f[U::N], g[U::N];
                    U::unpack(v[n], f);
                    U::unpack(z[j][n], g);
#pragma unroll
                    for (int i = 0; i < U::N; ++i) sum[j] = fmaf(f[i], g[i], sum[j]);
#pragma unroll
                    for (int i = 0; i < U::N; ++i) f[i] = __fmul_rn(f[i], c.weight);
                    if (u + n * t.threads < t.end && token_held(a, a.in[t.rank], token + (u + n * t.threads) * BYTES, BYTES, S) &&
                        row_of_expert_held(a, a.out[c.rank], at, BYTES, S))
                        U::store(at, U::pack(f));
                }
            }
        }
        // the team's sums: its warps', in order
#pragma unroll
        for (int j = 0; j < KB; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
            if (threadIdx.x % 32 == 0) parts[warp][j] = sum[j];
        }
        __syncthreads();
        if (t.on && t.thread < KB && first + t.thread < a.k) {
            float s = 0.0f;
            for (uint32_t w = 0; w < warps; ++w) s += parts[warp + w][t.thread];
            const uint64_t entry = uint64_t(t.token) * a.k + first + t.thread;
            if (entry_held(a, entry)) a.dweights[t.rank][entry] = t.list[first + t.thread].row ? s : 0.0f;
        }
        __syncthreads();
    }
}

template <typename T, int PM, int BYTES, int KB, int UN>
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
    // a team has about four units a thread, and more threads where there are few tokens or many choices
    const uint64_t units = N.hidden * elem_bytes(L.dtype) / BYTES, tokens = N.rows * uint64_t(L.p), sms = uint64_t(L.num_sms);
    a.team_shift = 5;
    while (a.team_shift < 8 && ((uint64_t(4 * UN) << a.team_shift) < units || tokens >> (8 - a.team_shift) < 4 * sms || N.k > 32)) ++a.team_shift;
    const uint32_t teams = kRowsThreads >> a.team_shift;
    const unsigned grid = unsigned((tokens + teams - 1) / teams);
    // few tokens: a row over several CTAs (the gradient's sums stay in one)
    uint64_t split = 1;
    if (N.op != ROWS_GRAD && grid < 4 * sms) {
        const uint64_t most = (units + kRowsThreads - 1) / kRowsThreads;
        split = (4 * sms + grid - 1) / grid;
        if (split > most) split = most;
        if (split < 1) split = 1;
    }
    const size_t smem = teams * N.k * sizeof(Choice);
    static std::atomic<unsigned long long> ready[3];
    void (*kern)(RowsArgs<PM>) = nullptr;
    if constexpr (std::is_same<T, I32>::value)
        kern = dispatch_kernel<T, PM, BYTES, 4>;
    else
        kern = N.op == ROWS_DISPATCH ? dispatch_kernel<T, PM, BYTES, 4> : N.op == ROWS_COMBINE ? combine_kernel<T, PM, BYTES, KB, UN> : combine_grad_kernel<T, PM, BYTES, KB, UN>;
    cudaError_t err = smem > 48 * 1024 ? allow_dynamic_smem(kern, 4096 * sizeof(Choice), L.device, ready[N.op]) : cudaSuccess;
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, unsigned(split));
    cfg.blockDim = dim3(kRowsThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kern, a);
    if (err != cudaSuccess) return err;
    info->kernel = N.op == ROWS_DISPATCH ? "expert_dispatch" : N.op == ROWS_COMBINE ? "expert_combine" : "expert_combine_grad";
    info->grid = int(grid * split);
    info->block = kRowsThreads;
    info->smem = smem;
    info->kernels = 1;
    return cudaSuccess;
}

// Units as wide as every address and the row allow, and batches by the number
// of choices.  Measured (graph replay, us; 16-byte units unless said; batches
// as choices x units):
//   combine, 8 x 4000 x 4096 bf16, k=2       2x4 102   2x2 106
//   combine's gradient, the same             2x4 160   2x2 162-170
//   gradient, 4 x 20000 x 512 f16, k=1       2x4 64    2x2 48: a row of 64 units fills two for each of 32 threads
//   gradient, 8 x 4000 x 2048 bf16, k=4      4x2 155
//   gradient, 2 x 4000 x 1002 f16, k=3       4-byte units, 8x4 27   4x2 30
//   gradient, 2 x 4000 x 1001 bf16, k=4      2-byte units, 8x4 104  4x2 94
//   combine, the same                        2-byte units, 8x4 52   4x2 36
// with the registers held to three CTAs an SM for 8 units of 16 bytes (four:
// 8 x 2048 x 7168 bf16, k=8, 602 and not 587) and to four for the others.
template <typename T, int PM>
static cudaError_t rows_width(const Launch &L, const RowsLaunch &N, LaunchInfo *info)
{
    constexpr bool wide = Traits<T>::VEC == 4;
    if (N.align >= 16) {
        if (PM > 8 || N.k > 4 || N.op == ROWS_DISPATCH) return rows_launch<T, PM, 16, 8, 1>(L, N, info);
        if constexpr (PM <= 8) {
            if (N.k > 2) return rows_launch<T, PM, 16, 4, 2>(L, N, info);
            return N.hidden < 128 * Traits<T>::VEC ? rows_launch<T, PM, 16, 2, 2>(L, N, info) : rows_launch<T, PM, 16, 2, 4>(L, N, info);
        }
    }
    if (wide || N.align >= 4) return rows_launch<T, PM, 4, 8, 4>(L, N, info);
    if constexpr (!wide) return rows_launch<T, PM, 2, 4, 2>(L, N, info);
    return cudaErrorInvalidValue;
}

template <typename T>
static cudaError_t rows_dtype(const Launch &L, const RowsLaunch &N, LaunchInfo *info)
{
    return L.p <= 8 ? rows_width<T, 8>(L, N, info) : rows_width<T, kMaxRanks>(L, N, info);
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
