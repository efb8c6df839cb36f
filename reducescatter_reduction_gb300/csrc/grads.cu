// The global norm of many gradient tensors, and their clipping by it.
//
//   norm = sqrt(sum x^2),  out = x min(1, max_norm / (norm + 1e-6))
// A tensor is cut into tiles of 16-byte groups that begin on 128-byte boundaries
// of memory wherever the tensor begins (on 16-byte boundaries a warp's
// loads go over 17 sectors, not 16: with that and the sums below, the norm of 300 bf16 tensors of 1.2 GB 190 -> 177 us); the tiles of all tensors are numbered
// through, and a CTA takes consecutive ones, so tensors of any size share the
// SMs evenly.  The tensors' addresses, and where every fourth share begins among them, travel as
// kernel parameters.  Bound by memory where the tensors are large: three
// passes over 300 bf16 tensors of 1.2 GB, out of place, in 553 us, 6.5 TB/s, in place in 547; below some MB by the
// launches and the join of the CTAs' sums (3 + 2 us for 1000 values).  A tensor whose `out` lies otherwise between 16-byte
// boundaries than its `in` is stored element by element: clipping alone 354 us, with out 2 or 8 bytes on 1520 to 1600 (400 f32
// tensors of 12 MB 4.7, 6.3).
#include "logits.cuh"

namespace ccl {

constexpr unsigned kSiteGrads = 13;
constexpr int kGradThreads = 256;
constexpr int kGradBatch = 4;                                    // groups a thread has of a tile
constexpr uint32_t kGradTile = kGradThreads * kGradBatch;        // groups of a tile
constexpr uint32_t kGradMaxGrid = 1280;
constexpr uint32_t kGradSteps = 4;
// Shares of the tiles, an SM: one CTA of the norm has each.  (us; 4 against 8 an SM: the norm of 400 f32 tensors of 12 MB 7.3, 10.3,
// of 20 bf16 ones of 100 MB 17.9, 20.5, of 300 of 1.2 GB 177, 179.)
constexpr uint32_t kGradShares = 4;
static_assert(kGradMaxGrid <= kMaxPartials, "");

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
    uint16_t start[kGradMaxGrid / kGradSteps];   // the tensor of the first tile of every fourth share
    uint32_t count, share, more;         // tiles of a share; one more for the first `more`
    uint32_t team_shift;                 // clipping: 2^team_shift CTAs have a share
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
    uintptr_t base;      // the 128-byte boundary at or below the tensor's begin
    uint64_t first;      // this thread's first group
    uint64_t n;
    uint32_t shift;      // elements between the boundary and the tensor
    uint4 v[kGradBatch];

    __device__ __forceinline__ bool whole(uint64_t g) const { return g * VEC >= shift && (g + 1) * VEC <= shift + n; }
    __device__ __forceinline__ bool inside(uint64_t at) const { return at >= shift && at < shift + n; }
    __device__ __forceinline__ GradGroups(const GradRecord &t, uint32_t tile, uint32_t short_by, unsigned *status)
    {
        base = uintptr_t(t.in) & ~uintptr_t(127);
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
            } else if (g * VEC < shift + n && (g + 1) * VEC > shift) {
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

// A sum and what its roundings left out (Knuth's two-sum): fp32 twice, as
// this GPU takes 16 cycles for a warp's fp64 addition.  (The norm of 400 f32
// tensors, 1000 tiles: with an fp64 sum in every thread 14.8 us, with these 10.3.)
struct Twofold {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float v)
    {
        const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b)));
        hi = s;
    }
    __device__ __forceinline__ void add(const Twofold &o)
    {
        add(o.hi);
        lo = __fadd_rn(lo, o.lo);
    }
};

// The sum of the squares of a thread's groups.  In fp32 where that loses
// nothing: squares below 2^-149 vanish, and those below 2^-126 lose digits, but
// beside a sum of 2^-100 neither is seen; sums up to 2^100, of 2^19 tiles and
// 2^8 threads, stay in range (2^40 elements are at most 2^28 tiles, over 608 CTAs).  Smaller and larger sums, infinities and NaN go
// through fp64, element by element, and into `rest`.
template <typename T>
__device__ __forceinline__ void grad_squares(const GradRecord &t, uint32_t tile, uint32_t short_by, unsigned *status, Twofold &sum, double &rest)
{
    using G = GradGroups<T>;
    const G g(t, tile, short_by, status);
    Pair part[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
    for (int i = 0; i < kGradBatch; ++i)
#pragma unroll
        for (int e = 0; e < Group<T>::PAIRS; ++e) {
            const Pair f = Group<T>::pair(g.v[i], e);
            part[e % 2] = fma(f, f, part[e % 2]);
        }
    const Pair both = part[0] + part[1];
    const float s = both.x + both.y;
    if (s >= 0x1p-100f && s <= 0x1p100f) {
        sum.add(s);
        return;
    }
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kGradBatch; ++i) any |= g.v[i].x | g.v[i].y | g.v[i].z | g.v[i].w;
    if ((any & (G::VEC == 4 ? 0x7fffffffu : 0x7fff7fffu)) == 0) return;       // zeros of either sign
#pragma unroll
    for (int i = 0; i < kGradBatch; ++i) {
        float f[G::VEC];
        Traits<T>::unpack(g.v[i], f);
#pragma unroll
        for (uint32_t e = 0; e < G::VEC; ++e) rest = ::fma(double(f[e]), double(f[e]), rest);
    }
}

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int CAP>
__global__ void __launch_bounds__(kGradThreads) grad_norm_kernel(const __grid_constant__ GradArgs<CAP> a)
{
    __shared__ bool last;
    grid_dependency_wait();
    grid_dependents_launch();
    const uint32_t begin = blockIdx.x * a.share + min(blockIdx.x, a.more), end = begin + a.share + (blockIdx.x < a.more ? 1 : 0);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    Twofold mine;
    double rest = 0.0;
    uint32_t i = a.start[blockIdx.x / kGradSteps];
    for (uint32_t tile = begin; tile < end; ++tile) {
        while (i + 1 < a.count && a.t[i + 1].first <= tile) ++i;
        const GradRecord &t = a.t[i];
        if (t.dtype == DT_F32) grad_squares<F32>(t, tile, a.short_by, a.status, mine, rest);
        else if (t.dtype == DT_F16) grad_squares<F16>(t, tile, a.short_by, a.status, mine, rest);
        else grad_squares<BF16>(t, tile, a.short_by, a.status, mine, rest);
    }
    // the CTA's sum, in a fixed order
    __shared__ Twofold part_s[kGradThreads / 32];
    __shared__ double rest_s[kGradThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Twofold other;
        other.hi = __shfl_xor_sync(0xffffffffu, mine.hi, o);
        other.lo = __shfl_xor_sync(0xffffffffu, mine.lo, o);
        mine.add(other);
    }
    if (__any_sync(0xffffffffu, rest != 0.0)) rest = warp_sum(rest);     // (NaN is not 0)
    if (lane == 0) {
        part_s[warp] = mine;
        rest_s[warp] = rest;
    }
    __syncthreads();
    double sum = 0.0;
    if (threadIdx.x == 0) {
        for (int w = 1; w < kGradThreads / 32; ++w) mine.add(part_s[w]);
        sum = double(mine.hi) + double(mine.lo);
        for (int w = 0; w < kGradThreads / 32; ++w)
            if (rest_s[w] != 0.0) sum += rest_s[w];
        last = true;
        if (gridDim.x > 1) {
            a.partials[blockIdx.x] = sum;
            __threadfence();
            last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
        }
    }
    if (gridDim.x > 1) {
        __syncthreads();
        if (!last) return;
        __threadfence();
        sum = 0.0;
        for (uint32_t b = threadIdx.x; b < gridDim.x; b += kGradThreads) sum += __ldcg(&a.partials[b]);
        sum = warp_sum(sum);
        if (lane == 0) rest_s[warp] = sum;
        __syncthreads();
        sum = 0.0;
        if (threadIdx.x == 0) {
            for (int w = 0; w < kGradThreads / 32; ++w) sum += rest_s[w];
            *a.ticket = 0;
        }
    }
    if (threadIdx.x == 0) {
        if (!a.first_launch) sum += *a.total;
        if (a.last_launch) a.norm[0] = float(sqrt(sum));
        else *a.total = sum;
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
    const uint32_t part = blockIdx.x >> a.team_shift, begin = part * a.share + min(part, a.more), end = begin + a.share + (part < a.more ? 1 : 0);
    if (begin == end) return;
    uint32_t i = a.start[part / kGradSteps];
    while (i + 1 < a.count && a.t[i + 1].first < end) ++i;
    // backwards: what the norm's pass read last is still in L2
    for (uint32_t at = blockIdx.x & ((1u << a.team_shift) - 1); at < end - begin; at += 1u << a.team_shift) {
        const uint32_t tile = end - 1 - at;
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
        const unsigned by = t.dtype == CCL_F32 ? 2 : 1;      // log2 of an element's bytes
        const uint64_t groups = (uintptr_t(t.in) % 128 + (t.n << by) + 15) >> 4;
        a.t[a.count++] = {t.in, t.out, t.n, uint32_t(tiles), uint32_t(t.dtype)};
        tiles += (groups + kGradTile - 1) / kGradTile;
    }
    while (*next < N.count && (N.tensors[*next].n == 0 || (N.tensors[*next].copy && !N.clip))) ++*next;
    a.max_norm = N.max_norm;
    a.first_launch = first;
    a.last_launch = *next == N.count;
    a.norm = N.norm;
    a.ticket = static_cast<unsigned *>(N.scratch);
    a.total = reinterpret_cast<double *>(static_cast<char *>(N.scratch) + 8);
    a.partials = reinterpret_cast<double *>(static_cast<char *>(N.scratch) + kScratchHead);
    a.status = L.status;
    a.short_by = L.stall_test == 2 ? 1 : 0;
    const uint64_t ctas = uint64_t(L.num_sms) * kGradShares, most = ctas < kGradMaxGrid ? ctas : kGradMaxGrid;
    const unsigned grid = unsigned(tiles < 1 ? 1 : tiles < most ? tiles : most);
    a.share = uint32_t(tiles / grid);
    a.more = uint32_t(tiles % grid);
    // Clipping, CTAs a share.  Measured (us for norm and clipping; 1 / 2 / 4 / 8): 370 tiles - / 9.9 / 10.0 / 11.1, 1000 tiles
    // - / 11.4 / 11.9 / 13.4, 12000 - / 49.4 / 49.1 / 49.3, 73000 614 / 587 / 557 / 552.
    a.team_shift = tiles <= grid ? 0 : a.share < 8 ? 1 : a.share < 32 ? 2 : 3;
    for (uint32_t b = 0, i = 0; b < grid; b += kGradSteps) {
        const uint32_t tile = b * a.share + (b < a.more ? b : a.more);
        while (i + 1 < a.count && a.t[i + 1].first <= tile) ++i;
        a.start[b / kGradSteps] = uint16_t(i);
    }
    const cudaError_t err = launch_dependent(N.clip ? grad_clip_kernel<CAP> : grad_norm_kernel<CAP>, N.clip ? grid << a.team_shift : grid, kGradThreads, 0, L.stream, a);
    if (err != cudaSuccess) return err;
    info->kernel = N.clip ? "grad_clip" : "grad_norm";
    info->grid = int(N.clip ? grid << a.team_shift : grid);
    info->block = kGradThreads;
    ++info->kernels;
    return cudaSuccess;
}

cudaError_t launch_grads(const Launch &L, const GradLaunch &N, LaunchInfo *info)
{
    size_t next = 0;
    bool first = true;
    do {
        const cudaError_t err = N.count <= 64    ? grad_launch<64>(L, N, &next, first, info)
                                : N.count <= 448 ? grad_launch<448>(L, N, &next, first, info)
                                                 : grad_launch<896>(L, N, &next, first, info);
        if (err != cudaSuccess) return err;
        first = false;
    } while (next < N.count);
    return cudaSuccess;
}

}  // namespace ccl
