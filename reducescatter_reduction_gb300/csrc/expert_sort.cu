// The rows of all ranks' choices in their experts' buffers: a stable counting
// sort by expert.
//
// The choices of all ranks, in the order (rank, token, choice), are cut into
// parts, one a CTA.  A first kernel counts each part's choices by expert; the
// second adds up the counts of the parts before its own, which gives where
// the part's choices of each expert begin, and numbers them: a warp takes a
// stretch of the part, counts it, and walks through it 32 choices at a time,
// a choice's number being the warp's begin plus the lanes before it with the
// same expert.  All sums are of integers, and the order is fixed.
#include <algorithm>

#include "logits.cuh"

namespace ccl {

constexpr unsigned kSiteSort = 12;
constexpr int kSortThreads = 1024;
constexpr uint32_t kSortSmem = 160 * 1024;   // of the warps' counters

template <int PM>
struct SortArgs {
    const int32_t *ids[PM];
    const uint8_t *valid[PM];
    int32_t *slots[PM];
    int32_t *offsets, *cells;      // cells: [parts, experts]
    uint32_t rows, p, k, experts, capacity, all, per_rank;   // all: choices of all ranks
    uint32_t parts, part;          // choices of a part
    uint32_t q, rem;               // experts of a rank: q + 1 for the first rem, then q
    uint32_t warps;                // warps that number choices
    int has_valid;
    FastDiv by_k, by_rank, by_q1, by_q;
    // checked build:
    unsigned *status;
    uint32_t held;                 // rows that every list has
};

// The expert of choice g, or `experts` if it has none.
template <int PM>
__device__ __forceinline__ uint32_t expert_of(const SortArgs<PM> &a, uint32_t g)
{
    const uint32_t r = div_by(g, a.by_rank), at = g - r * a.per_rank, row = div_by(at, a.by_k);
    if (!in_bounds(row < a.held, a.status, kSiteSort, at)) return a.experts;
    const uint32_t e = uint32_t(a.ids[r][at]);
    if (a.has_valid && !a.valid[r][row]) return a.experts;
    return min(e, a.experts);
}

template <int PM>
__device__ __forceinline__ uint32_t first_expert(const SortArgs<PM> &a, uint32_t r) { return r * a.q + min(r, a.rem); }
template <int PM>
__device__ __forceinline__ uint32_t rank_of_expert(const SortArgs<PM> &a, uint32_t e)
{
    const uint32_t big = a.rem * (a.q + 1);
    return e < big ? div_by(e, a.by_q1) : a.rem + div_by(e - big, a.by_q);
}

template <int PM>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const __grid_constant__ SortArgs<PM> a)
{
    extern __shared__ uint32_t hist[];
    for (uint32_t e = threadIdx.x; e < a.experts; e += kSortThreads) hist[e] = 0;
    grid_dependency_wait();
    grid_dependents_launch();
    __syncthreads();
    const uint32_t begin = blockIdx.x * a.part, end = min(a.all, begin + a.part);
    for (uint32_t g = begin + threadIdx.x; g < end; g += kSortThreads) {
        const uint32_t e = expert_of(a, g);
        if (e < a.experts) atomicAdd(&hist[e], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.experts; e += kSortThreads) {
        const uint64_t cell = uint64_t(blockIdx.x) * a.experts + e;
        if (in_bounds(cell < kSortCells, a.status, kSiteSort, cell)) a.cells[cell] = int32_t(hist[e]);
    }
}

template <int PM>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const __grid_constant__ SortArgs<PM> a)
{
    extern __shared__ uint32_t smem[];
    const uint32_t E = a.experts, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t *begin_s = smem;            // [E] choices of an expert before the part, then where they begin in the rank's buffer
    uint32_t *total_s = smem + E;        // [E + 1] choices before an expert's, over all experts
    uint32_t *count_s = total_s + E + 1; // [warps, E]
    __shared__ uint32_t carry_s, warp_s[32];
    for (uint32_t i = threadIdx.x; i < a.warps * E; i += kSortThreads) count_s[i] = 0;
    grid_dependency_wait();
    grid_dependents_launch();
    for (uint32_t e = threadIdx.x; e < E; e += kSortThreads) {
        uint32_t before = 0, total = 0;
#pragma unroll 8
        for (uint32_t b = 0; b < a.parts; ++b) {
            const uint64_t cell = uint64_t(b) * E + e;
            const uint32_t n = in_bounds(cell < kSortCells, a.status, kSiteSort, cell) ? uint32_t(a.cells[cell]) : 0u;
            before += b < blockIdx.x ? n : 0u;
            total += n;
        }
        begin_s[e] = before;
        total_s[e] = total;
    }
    if (threadIdx.x == 0) carry_s = 0;
    __syncthreads();
    // exclusive sums of the totals, 1024 experts at a time
    for (uint32_t first = 0; first < E; first += kSortThreads) {
        const uint32_t e = first + threadIdx.x;
        const uint32_t n = e < E ? total_s[e] : 0;
        uint32_t up = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= uint32_t(o)) up += v;
        }
        if (lane == 31) warp_s[warp] = up;
        __syncthreads();
        if (warp == 0) {
            uint32_t w = warp_s[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= uint32_t(o)) w += v;
            }
            warp_s[lane] = w;
        }
        __syncthreads();
        const uint32_t carry = carry_s;
        if (e < E) total_s[e] = carry + up - n + (warp ? warp_s[warp - 1] : 0);
        __syncthreads();
        if (threadIdx.x == 0) carry_s = carry + warp_s[31];
        __syncthreads();
    }
    if (threadIdx.x == 0) total_s[E] = carry_s;
    __syncthreads();
    if (blockIdx.x == 0) {
        // rank r's part: begins of its experts and their end
        for (uint32_t i = threadIdx.x; i < E; i += kSortThreads) {
            const uint32_t r = rank_of_expert(a, i);
            a.offsets[i + r] = int32_t(min(total_s[i] - total_s[first_expert(a, r)], a.capacity));
        }
        for (uint32_t r = threadIdx.x; r < a.p; r += kSortThreads) {
            const uint32_t from = first_expert(a, r), to = first_expert(a, r + 1);
            a.offsets[to + r] = int32_t(min(total_s[to] - total_s[from], a.capacity));
        }
    }
    for (uint32_t e = threadIdx.x; e < E; e += kSortThreads) begin_s[e] += total_s[e] - total_s[first_expert(a, rank_of_expert(a, e))];
    // the warps' stretches of the part
    const uint32_t part_end = min(uint64_t(a.all), (uint64_t(blockIdx.x) + 1) * a.part);
    const uint32_t stretch = (a.part / 32 + a.warps - 1) / a.warps * 32;
    const uint64_t from = uint64_t(blockIdx.x) * a.part + uint64_t(warp) * stretch;
    const uint32_t begin = uint32_t(min(uint64_t(part_end), from)), end = uint32_t(min(uint64_t(part_end), from + stretch));
    uint32_t *mine = count_s + warp * E;
    if (warp < a.warps)
        for (uint32_t g = begin + lane; g < end; g += 32) {
            const uint32_t e = expert_of(a, g);
            if (e < E) atomicAdd(&mine[e], 1u);
        }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < E; e += kSortThreads) {
        uint32_t at = begin_s[e];
        for (uint32_t w = 0; w < a.warps; ++w) {
            const uint32_t n = count_s[w * E + e];
            count_s[w * E + e] = at;
            at += n;
        }
    }
    __syncthreads();
    if (warp >= a.warps) return;
    for (uint32_t g0 = begin; g0 < end; g0 += 32) {
        const uint32_t g = g0 + lane;
        const uint32_t e = g < end ? expert_of(a, g) : E;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        uint32_t at = 0;
        if (e < E) at = mine[e] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (e < E && lane == 31 - __clz(same)) mine[e] = at + 1;
        __syncwarp();
        if (g < end) {
            const uint32_t r = div_by(g, a.by_rank), i = g - r * a.per_rank;
            int32_t slot = -1;
            if (e < E && at < a.capacity) slot = int32_t(rank_of_expert(a, e) * a.capacity + at);
            if (in_bounds(i < a.held * a.k, a.status, kSiteSort, i)) a.slots[r][i] = slot;
        }
    }
}

template <int PM>
static cudaError_t sort_launch(const Launch &L, const SortLaunch &N, LaunchInfo *info)
{
    SortArgs<PM> a = {};
    for (int r = 0; r < L.p && N.rows; ++r) {
        a.ids[r] = N.ids[r];
        a.valid[r] = N.valid ? N.valid[r] : nullptr;
        a.slots[r] = N.slots[r];
    }
    a.offsets = N.offsets;
    a.cells = N.cells;
    a.rows = uint32_t(N.rows);
    a.p = uint32_t(L.p);
    a.k = N.k;
    a.experts = N.experts;
    a.capacity = N.capacity;
    a.per_rank = a.rows * a.k;
    a.all = a.per_rank * a.p;
    // a part: a multiple of 32 choices; as many parts as SMs, or as the cells hold
    uint32_t parts = std::min<uint32_t>(std::min<uint32_t>(unsigned(L.num_sms), kSortCells / a.experts), (a.all + 2047) / 2048);
    if (parts < 1) parts = 1;
    a.part = uint32_t((uint64_t(a.all) + parts - 1) / parts + 31) / 32 * 32;
    if (a.part == 0) a.part = 32;
    a.parts = std::max<uint32_t>(1, (a.all + a.part - 1) / a.part);
    a.q = a.experts / a.p;
    a.rem = a.experts % a.p;
    a.warps = std::min<uint32_t>(kSortThreads / 32, kSortSmem / (a.experts * 4));
    a.has_valid = N.valid ? 1 : 0;
    a.by_k = fast_div(a.k);
    a.by_rank = fast_div(a.per_rank ? a.per_rank : 1);
    a.by_q1 = fast_div(a.q + 1);
    a.by_q = fast_div(a.q ? a.q : 1);
    a.status = L.status;
    a.held = a.rows - (L.stall_test == 2 && a.rows ? 1 : 0);
    static std::atomic<unsigned long long> ready{0};
    const size_t smem = (size_t(a.experts) * (a.warps + 2) + 1) * 4;
    cudaError_t err = allow_dynamic_smem(sort_place_kernel<PM>, kSortSmem + (2 * 4096 + 1) * 4, L.device, ready);
    if (err != cudaSuccess) return err;
    err = launch_dependent(sort_count_kernel<PM>, a.parts, kSortThreads, a.experts * 4, L.stream, a);
    if (err != cudaSuccess) return err;
    info->kernel = "expert_sort";
    info->grid = int(a.parts);
    info->block = kSortThreads;
    info->smem = smem;
    info->kernels = 1;
    err = launch_dependent(sort_place_kernel<PM>, a.parts, kSortThreads, smem, L.stream, a);
    if (err == cudaSuccess) info->kernels = 2;
    return err;
}

cudaError_t launch_expert_sort(const Launch &L, const SortLaunch &N, LaunchInfo *info)
{
    return L.p <= 8 ? sort_launch<8>(L, N, info) : sort_launch<kMaxRanks>(L, N, info);
}

}  // namespace ccl
