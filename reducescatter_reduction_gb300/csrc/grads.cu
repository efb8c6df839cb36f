// The global norm of many gradient tensors, and their clipping by it.
//
//   norm = sqrt(sum x^2),  out = x min(1, max_norm / (norm + 1e-6))
// A tensor is cut into tiles of 16-byte groups that lie on 16-byte boundaries
// of memory wherever the tensor begins; the tiles of all tensors are numbered
// through, and a CTA takes consecutive ones, so tensors of any size share the
// SMs evenly.  The tensors' addresses travel as kernel parameters.
#include "logits.cuh"

namespace ccl {

constexpr unsigned kSiteGrads = 13;
constexpr int kGradThreads = 256;
constexpr int kGradBatch = 4;                                    // groups a thread has of a tile
constexpr uint32_t kGradTile = kGradThreads * kGradBatch;        // groups of a tile

struct GradRecord {
    const void *in;
    void *out;
    uint64_t n;
    uint32_t first;      // its first tile
    uint32_t dtype;
};

template <int CAP>
struct GradArgs {
    GradRecord t[CAP];
    uint32_t count, tiles;
    float max_norm;
    int first_launch, last_launch;
    float *norm;
    unsigned *ticket;
    double *total;       // over the launches of a call
    double *partials;
    // checked build:
    unsigned *status;
    uint32_t short_by;   // elements that the checks take every tensor to lack (debug hook)
};

__device__ __forceinline__ bool grad_held(const void *buf, uint64_t n, const void *at, uint32_t bytes, uint32_t S, uint32_t short_by, unsigned *status)
{
    return !kBoundsCheck || in_buffer(at, bytes, buf, (n - short_by) * S, status, kSiteGrads);
}

// The groups of a tile that are this thread's: full ones are loaded whole, of
// others the tensor's own elements; what lies outside is zero.
template <typename T>
struct GradGroups {
    using Tr = Traits<T>;
    static constexpr uint32_t VEC = Tr::VEC, S = 16 / VEC;
    uintptr_t base;      // the boundary at or below the tensor's begin
    uint64_t first;      // this thread's first group
    uint64_t n;
    uint32_t shift;      // elements between the boundary and the tensor
    uint4 v[kGradBatch];

    __device__ __forceinline__ bool whole(uint64_t g) const { return g * VEC >= shift && (g + 1) * VEC <= shift + n; }
    __device__ __forceinline__ bool inside(uint64_t at) const { return at >= shift && at < shift + n; }
    __device__ __forceinline__ GradGroups(const GradRecord &t, uint32_t tile, uint32_t short_by, unsigned *status)
    {
        base = uintptr_t(t.in) & ~uintptr_t(15);
        shift = uint32_t(uintptr_t(t.in) - base) / S;
        n = t.n;
        first = uint64_t(tile - t.first) * kGradTile + threadIdx.x;
#pragma unroll
        for (int i = 0; i < kGradBatch; ++i) {
            const uint64_t g = first + i * kGradThreads;
            v[i] = make_uint4(0, 0, 0, 0);
            const char *at = reinterpret_cast<const char *>(base) + g * 16;
            if (whole(g)) {
                if (grad_held(t.in, n, at, 16, S, short_by, status)) v[i] = ld_coherent_v4(at);
            } else if (g * VEC < shift + n) {
                float f[VEC];
#pragma unroll
                for (uint32_t e = 0; e < VEC; ++e) {
                    f[e] = 0.0f;
                    if (inside(g * VEC + e) && grad_held(t.in, n, at + e * S, S, S, short_by, status)) f[e] = Tr::load1(at, e);
                }
                v[i] = Tr::pack(f);
            }
        }
    }
};

// The sum of the squares of a thread's groups.  In fp32 where that loses
// nothing: squares below 2^-149 vanish, and those below 2^-126 lose digits, but
// beside a sum of 2^-80 neither is seen.  Smaller and larger sums, infinities and NaN go through fp64,
// element by element.
template <typename T>
__device__ __forceinline__ double grad_squares(const GradRecord &t, uint32_t tile, uint32_t short_by, unsigned *status)
{
    using G = GradGroups<T>;
    const G g(t, tile, short_by, status);
    float part[kGradBatch];
#pragma unroll
    for (int i = 0; i < kGradBatch; ++i) {
        float f[G::VEC];
        Traits<T>::unpack(g.v[i], f);
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (uint32_t e = 0; e < G::VEC; e += 2) {
            a = fmaf(f[e], f[e], a);
            b = fmaf(f[e + 1], f[e + 1], b);
        }
        part[i] = a + b;
    }
    const float s = (part[0] + part[1]) + (part[2] + part[3]);
    if (s >= 0x1p-80f && s <= 0x1p126f) return double(s);
    double d = 0.0;
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kGradBatch; ++i) any |= g.v[i].x | g.v[i].y | g.v[i].z | g.v[i].w;
    if (any == 0) return d;
#pragma unroll
    for (int i = 0; i < kGradBatch; ++i) {
        float f[G::VEC];
        Traits<T>::unpack(g.v[i], f);
#pragma unroll
        for (uint32_t e = 0; e < G::VEC; ++e) d = ::fma(double(f[e]), double(f[e]), d);
    }
    return d;
}

// The tensor that has a tile.
template <int CAP>
__device__ __forceinline__ uint32_t grad_tensor(const GradArgs<CAP> &a, uint32_t tile)
{
    uint32_t lo = 0, hi = a.count;      // t[lo].first <= tile < t[hi].first
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (a.t[mid].first <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double red[kGradThreads / 32];
    __syncthreads();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < kGradThreads / 32; ++w) v += red[w];
    return v;
}

template <int CAP>
__global__ void __launch_bounds__(kGradThreads) grad_norm_kernel(const __grid_constant__ GradArgs<CAP> a)
{
    __shared__ bool last;
    grid_dependency_wait();
    grid_dependents_launch();
    const uint32_t begin = uint32_t(uint64_t(a.tiles) * blockIdx.x / gridDim.x), end = uint32_t(uint64_t(a.tiles) * (blockIdx.x + 1) / gridDim.x);
    double sum = 0.0;
    uint32_t i = begin < end ? grad_tensor(a, begin) : 0;
    for (uint32_t tile = begin; tile < end; ++tile) {
        while (i + 1 < a.count && a.t[i + 1].first <= tile) ++i;
        const GradRecord &t = a.t[i];
        sum += t.dtype == DT_F32 ? grad_squares<F32>(t, tile, a.short_by, a.status) : t.dtype == DT_F16 ? grad_squares<F16>(t, tile, a.short_by, a.status)
                                                                                               : grad_squares<BF16>(t, tile, a.short_by, a.status);
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        a.partials[blockIdx.x] = sum;
        __threadfence();
        last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    sum = 0.0;
    for (uint32_t b = threadIdx.x; b < gridDim.x; b += kGradThreads) sum += __ldcg(&a.partials[b]);
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        if (!a.first_launch) sum += *a.total;
        if (a.last_launch) a.norm[0] = float(sqrt(sum));
        else *a.total = sum;
        *a.ticket = 0;
    }
}

template <typename T>
__device__ __forceinline__ void grad_scale(const GradRecord &t, uint32_t tile, float factor, uint32_t short_by, unsigned *status)
{
    using G = GradGroups<T>;
    using Tr = Traits<T>;
    const G g(t, tile, short_by, status);
    const bool together = ((uintptr_t(t.out) - uintptr_t(t.in)) & 15) == 0;
    char *to = static_cast<char *>(t.out) - int64_t(g.shift) * G::S;     // where `base` goes
#pragma unroll
    for (int i = 0; i < kGradBatch; ++i) {
        const uint64_t at = g.first + i * kGradThreads;
        float f[G::VEC];
        Tr::unpack(g.v[i], f);
#pragma unroll
        for (uint32_t e = 0; e < G::VEC; ++e) f[e] = __fmul_rn(f[e], factor);
        if (together && g.whole(at)) {
            if (grad_held(t.out, g.n, to + at * 16, 16, G::S, short_by, status)) st_stream_v4(to + at * 16, Tr::pack(f));
        } else {
#pragma unroll
            for (uint32_t e = 0; e < G::VEC; ++e)
                if (g.inside(at * G::VEC + e) && grad_held(t.out, g.n, to + at * 16 + e * G::S, G::S, G::S, short_by, status))
                    Tr::store1(to + at * 16, e, f[e]);
        }
    }
}

template <int CAP>
__global__ void __launch_bounds__(kGradThreads) grad_clip_kernel(const __grid_constant__ GradArgs<CAP> a)
{
    grid_dependency_wait();
    grid_dependents_launch();
    const float by = __fdiv_rn(a.max_norm, a.norm[0] + 1e-6f);
    const float factor = by > 1.0f ? 1.0f : by;                  // (NaN stays NaN)
    if (a.last_launch && blockIdx.x == 0 && threadIdx.x == 0) a.norm[1] = factor;
    const uint32_t begin = uint32_t(uint64_t(a.tiles) * blockIdx.x / gridDim.x), end = uint32_t(uint64_t(a.tiles) * (blockIdx.x + 1) / gridDim.x);
    if (begin == end) return;
    uint32_t i = grad_tensor(a, end - 1);
    // backwards: what the norm's pass read last is still in L2
    for (uint32_t tile = end; tile-- > begin;) {
        while (a.t[i].first > tile) --i;
        const GradRecord &t = a.t[i];
        if (factor == 1.0f && t.out == t.in) continue;
        if (t.dtype == DT_F32) grad_scale<F32>(t, tile, factor, a.short_by, a.status);
        else if (t.dtype == DT_F16) grad_scale<F16>(t, tile, factor, a.short_by, a.status);
        else grad_scale<BF16>(t, tile, factor, a.short_by, a.status);
    }
}

template <int CAP>
static cudaError_t grad_launch(const Launch &L, const GradLaunch &N, size_t *next, bool first, LaunchInfo *info)
{
    GradArgs<CAP> a;
    a.count = 0;
    uint64_t tiles = 0;
    for (; *next < N.count && a.count < CAP; ++*next) {
        const ccl_tensor_t &t = N.tensors[*next];
        if (t.n == 0 || (t.copy && !N.clip)) continue;
        const uint32_t S = uint32_t(elem_bytes(t.dtype)), vec = 16 / S;
        const uint64_t groups = (uintptr_t(t.in) % 16 / S + t.n + vec - 1) / vec;
        a.t[a.count++] = {t.in, t.out, t.n, uint32_t(tiles), uint32_t(t.dtype)};
        tiles += (groups + kGradTile - 1) / kGradTile;
    }
    while (*next < N.count && (N.tensors[*next].n == 0 || (N.tensors[*next].copy && !N.clip))) ++*next;
    a.tiles = uint32_t(tiles);
    a.max_norm = N.max_norm;
    a.first_launch = first;
    a.last_launch = *next == N.count;
    a.norm = N.norm;
    a.ticket = static_cast<unsigned *>(N.scratch);
    a.total = reinterpret_cast<double *>(static_cast<char *>(N.scratch) + 8);
    a.partials = reinterpret_cast<double *>(static_cast<char *>(N.scratch) + kScratchHead);
    a.status = L.status;
    a.short_by = L.stall_test == 2 ? 1 : 0;
    const uint64_t most = uint64_t(L.num_sms) * 8 < kMaxPartials ? uint64_t(L.num_sms) * 8 : kMaxPartials;
    const unsigned grid = unsigned(tiles < 1 ? 1 : tiles < most ? tiles : most);
    const cudaError_t err = launch_dependent(N.clip ? grad_clip_kernel<CAP> : grad_norm_kernel<CAP>, grid, kGradThreads, 0, L.stream, a);
    if (err != cudaSuccess) return err;
    info->kernel = N.clip ? "grad_clip" : "grad_norm";
    info->grid = int(grid);
    info->block = kGradThreads;
    ++info->kernels;
    return cudaSuccess;
}

cudaError_t launch_grads(const Launch &L, const GradLaunch &N, LaunchInfo *info)
{
    size_t next = 0;
    bool first = true;
    do {
        const cudaError_t err = N.count <= 64 ? grad_launch<64>(L, N, &next, first, info) : grad_launch<896>(L, N, &next, first, info);
        if (err != cudaSuccess) return err;
        first = false;
    } while (next < N.count);
    return cudaSuccess;
}

}  // namespace ccl
