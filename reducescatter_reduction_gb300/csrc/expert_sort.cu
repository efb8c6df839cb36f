// The rows of all ranks' choices in their experts' buffers: a stable counting
// sort by expert.
//
// The choices of all ranks, in the order (rank, token, choice), are cut into
// parts, one a CTA.  A first kernel counts each part's choices by expert; the
// second adds up the counts of the parts before its own, which gives where
// the part's choices of each expert begin, and numbers them: a warp takes a
// stretch of the part and walks through it 32 choices at a time.  A choice's
// number among its expert's in the stretch is what the warp has counted so
// far plus the lanes before it with the same expert; those are found by a
// ballot for each bit of the expert's number (match.any takes a step for each
// different expert among the lanes: with it 1 Mi choices of 256 experts on 8 ranks took 21.8 us, with ballots, and quads of cells
// in the sums, 17.6 then).
// All sums are of integers, and the order is fixed.  Bound by instructions and
// latency: 1 Mi choices of 256 experts on 8 ranks, 12.6 MB moved, take 15.5 us (padded 17.9; of 8 experts 13.1, of 512 18.2, of
// 4096 67, whose counters leave 9 warps and 64 parts), 2 Mi 27.5, 8 Mi 79, where numbers pass through the slots (200 MB):
// two launches, and in each CTA a chain of loads, ballots, sums and barriers.
#include <algorithm>

#include "logits.cuh"

namespace ccl {

constexpr unsigned kSiteSort = 12;
constexpr int kSortThreads = 1024;
constexpr uint32_t kSortSmem = 160 * 1024;   // of the warps' counters
constexpr int kSortItems = 8;                // choices a thread reads at once
// Up to this many choices one CTA counts and numbers them, in one launch, whose host time a second one would nearly double.
// Measured (256 experts, graph replay, us; one CTA against two kernels): 512 choices 4.6; 4096 7.0, 6.6; 8192 10.6, 6.8.
constexpr uint32_t kSortAlone = 4096;
// Choices of a part, at least: a part takes about 0.4 us for each 1024 of them, and every part more makes the sums before it
// longer (256 experts, us, with 512 and 2048: 8192 choices 6.8, 8.3; 65536 9.4, 9.0; 1 Mi has 6900 for each SM with either).
constexpr uint32_t kSortPart = 512;

template <int PM>
struct SortArgs {
    const int32_t *ids[PM];
    const uint8_t *valid[PM];
    int32_t *slots[PM];
    int32_t *offsets, *cells;      // cells: [parts, stride]
    uint32_t rows, p, k, experts, capacity, all, per_rank;   // all: choices of all ranks
    uint32_t parts, part;          // choices of a part
    uint32_t q, rem;               // experts of a rank: q + 1 for the first rem, then q
    uint32_t warps;                // warps that number choices
    uint32_t stride;               // of a part's cells: experts, up to a multiple of 4
    int has_valid;
    FastDiv by_k, by_rank, by_q1, by_q;
    // checked build:
    unsigned *status;
    uint32_t held;                 // rows that every list has
};

// Choices [begin, end), mostly of one rank: then its lists are taken once.
template <int PM>
struct Stretch {
    const SortArgs<PM> &a;
    uint32_t begin, end, rank, first;      // first: the rank's first choice
    bool one;
    __device__ __forceinline__ Stretch(const SortArgs<PM> &args, uint32_t b, uint32_t e) : a(args), begin(b), end(e)
    {
        rank = div_by(b, a.by_rank);
        first = rank * a.per_rank;
        one = e <= first + a.per_rank;
    }
    __device__ __forceinline__ uint32_t rank_of(uint32_t g) const { return one ? rank : div_by(g, a.by_rank); }
    // The expert of choice g, or `experts` if it has none.
    __device__ __forceinline__ uint32_t expert(uint32_t g) const
    {
        const uint32_t r = rank_of(g), at = g - (one ? first : r * a.per_rank);
        if (!in_bounds(at < a.held * a.k, a.status, kSiteSort, at)) return a.experts;
        const uint32_t e = uint32_t(a.ids[r][at]);
        if (a.has_valid && !a.valid[r][div_by(at, a.by_k)]) return a.experts;
        return min(e, a.experts);
    }
    // The experts of N choices of a thread, `step` apart; all loads go out at once.
    template <int N>
    __device__ __forceinline__ void experts(uint32_t g, uint32_t step, uint32_t (&e)[N]) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = g + i * step < end ? expert(g + i * step) : a.experts;
    }
    // Where the slot of choice g goes; null: nowhere (checked build).
    __device__ __forceinline__ int32_t *slot(uint32_t g) const
    {
        const uint32_t r = rank_of(g), at = g - (one ? first : r * a.per_rank);
        return in_bounds(at < a.held * a.k, a.status, kSiteSort, at) ? a.slots[r] + at : nullptr;
    }
};

template <int PM>
__device__ __forceinline__ uint32_t first_expert(const SortArgs<PM> &a, uint32_t r) { return r * a.q + min(r, a.rem); }
template <int PM>
__device__ __forceinline__ uint32_t rank_of_expert(const SortArgs<PM> &a, uint32_t e)
{
    const uint32_t big = a.rem * (a.q + 1);
    return e < big ? div_by(e, a.by_q1) : a.rem + div_by(e - big, a.by_q);
}

// A part's choices by expert, into the cells.
template <int PM>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const __grid_constant__ SortArgs<PM> a)
{
    extern __shared__ uint32_t hist[];
    for (uint32_t e = threadIdx.x; e < a.experts; e += kSortThreads) hist[e] = 0;
    grid_dependency_wait();
    grid_dependents_launch();
    __syncthreads();
    const uint32_t begin = blockIdx.x * a.part;
    const Stretch<PM> part(a, begin, min(a.all, begin + a.part));
    for (uint32_t g = begin + threadIdx.x; g < part.end; g += kSortThreads * kSortItems) {
        uint32_t e[kSortItems];
        part.experts(g, kSortThreads, e);
#pragma unroll
        for (int i = 0; i < kSortItems; ++i)
            if (e[i] < a.experts) atomicAdd(&hist[e[i]], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.stride; e += kSortThreads) {
        const uint64_t cell = uint64_t(blockIdx.x) * a.stride + e;
        if (in_bounds(cell < kSortCells, a.status, kSiteSort, cell)) a.cells[cell] = e < a.experts ? int32_t(hist[e]) : 0;
    }
}

// Exclusive sums of `of` [n], in place; of[n] receives the total.
__device__ __forceinline__ void scan_shared(uint32_t *of, uint32_t n)
{
    __shared__ uint32_t warp_s[32];
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t carry = 0;
    for (uint32_t first = 0; first < n; first += kSortThreads) {
        const uint32_t i = first + threadIdx.x, own = i < n ? of[i] : 0;
        uint32_t up = own;
#pragma unroll
        for (uint32_t o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o) up += v;
        }
        __syncthreads();
        if (lane == 31) warp_s[warp] = up;
        __syncthreads();
        uint32_t w = warp_s[lane];          // every warp adds up the warps for itself
#pragma unroll
        for (uint32_t o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += v;
        }
        const uint32_t before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0), all = __shfl_sync(0xffffffffu, w, 31);
        if (i < n) of[i] = carry + up - own + (warp ? before : 0);
        carry += all;
    }
    if (threadIdx.x == 0) of[n] = carry;
    __syncthreads();
}

// Numbers a part's choices.  ALONE: there is one part, and its counts are all there are.  BITS: at least those of experts - 1.
template <int PM, bool ALONE, int BITS>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const __grid_constant__ SortArgs<PM> a)
{
    extern __shared__ uint32_t smem[];
    const uint32_t E = a.experts, row = E + 1, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t *begin_s = smem;            // [E] choices of an expert before the part, then where they begin in the rank's buffer
    uint32_t *total_s = smem + E;        // [E + 1] choices of an expert, then those before an expert's
    uint32_t *count_s = total_s + E + 1; // [warps, E + 1] of an expert in a warp's stretch, then in those before it
    for (uint32_t i = threadIdx.x; i < 2 * E + 1 + a.warps * row; i += kSortThreads) smem[i] = 0;
    grid_dependency_wait();
    grid_dependents_launch();
    __syncthreads();
    // the warps' stretches of the part
    const uint32_t part_end = uint32_t(min(uint64_t(a.all), (uint64_t(blockIdx.x) + 1) * a.part));
    const uint32_t stretch = (a.part / 32 + a.warps - 1) / a.warps * 32;
    const uint64_t from = uint64_t(blockIdx.x) * a.part + uint64_t(warp) * stretch;
    const uint32_t begin = warp < a.warps ? uint32_t(min(uint64_t(part_end), from)) : part_end;
    const uint32_t end = warp < a.warps ? uint32_t(min(uint64_t(part_end), from + stretch)) : part_end;
    const Stretch<PM> part(a, begin, end);
    uint32_t *mine = count_s + warp * row;
    const bool kept = end - begin <= 32 * kSortItems;      // the stretch stays in registers; of others the numbers go through the slots
    uint32_t e[kSortItems], number[kSortItems];
    part.experts(begin + lane, 32, e);      // (under way while the cells are summed)
    if (!ALONE) {
        // Four experts a load; threads side by side take experts, and then shares of the parts, so that the loads of all
        // parts are under way at once.
        const uint32_t quads = a.stride / 4, shares = kSortThreads / quads, share = threadIdx.x / quads, x = (threadIdx.x - share * quads) * 4;
        const uint32_t b1 = a.parts * (share + 1) / shares;
        if (share < shares) {
            uint4 before = make_uint4(0, 0, 0, 0), total = before;
#pragma unroll 16
            for (uint32_t b = a.parts * share / shares; b < b1; ++b) {
                const uint64_t cell = uint64_t(b) * a.stride + x;
                if (!in_bounds(cell + 4 <= kSortCells, a.status, kSiteSort, cell)) continue;
                const uint4 n = *reinterpret_cast<const uint4 *>(a.cells + cell);
                total = make_uint4(total.x + n.x, total.y + n.y, total.z + n.z, total.w + n.w);
                if (b < blockIdx.x) before = make_uint4(before.x + n.x, before.y + n.y, before.z + n.z, before.w + n.w);
            }
            const uint32_t of[2][4] = {{before.x, before.y, before.z, before.w}, {total.x, total.y, total.z, total.w}};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (x + i < E) {
                    atomicAdd(&begin_s[x + i], of[0][i]);
                    atomicAdd(&total_s[x + i], of[1][i]);
                }
        }
    }
    for (uint32_t g0 = begin; g0 < end; g0 += 32 * kSortItems) {
        if (g0 != begin) part.experts(g0 + lane, 32, e);
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            if (g0 + i * 32 >= end) break;
            uint32_t same = __ballot_sync(0xffffffffu, e[i] < E);
#pragma unroll
            for (int b = 0; b < BITS; ++b) {
                const int set = int(e[i] << (31 - b)) >> 31;       // all ones or none
                same &= ~(__ballot_sync(0xffffffffu, set) ^ uint32_t(set));
            }
            number[i] = e[i] < E ? mine[e[i]] + __popc(same & ((1u << lane) - 1)) : 0;
            __syncwarp();
            if (e[i] < E && lane == 31 - __clz(same)) mine[e[i]] = number[i] + 1;
            __syncwarp();
            if (!kept && g0 + i * 32 + lane < end)
                if (int32_t *to = part.slot(g0 + i * 32 + lane)) *to = int32_t(number[i]);
        }
    }
    __syncthreads();
    // a warp takes an expert at a time, a lane a warp's count
#pragma unroll 4
    for (uint32_t x = warp; x < E; x += kSortThreads / 32) {
        const uint32_t own = lane < a.warps ? count_s[lane * row + x] : 0;
        uint32_t up = own;
#pragma unroll
        for (uint32_t o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o) up += v;
        }
        if (lane < a.warps) count_s[lane * row + x] = up - own;
        if (ALONE && lane == 31) total_s[x] = up;
    }
    __syncthreads();
    scan_shared(total_s, E);
    // begin_s: the slot of the part's first choice of an expert; end_s: the end of its rank's slots
    uint32_t *end_s = total_s;
    uint32_t at[4096 / kSortThreads], rank[4096 / kSortThreads];
#pragma unroll
    for (int i = 0; i < 4096 / kSortThreads; ++i) {
        const uint32_t x = threadIdx.x + i * kSortThreads;
        if (x >= E) break;
        rank[i] = rank_of_expert(a, x);
        at[i] = total_s[x] - total_s[first_expert(a, rank[i])];
        begin_s[x] += rank[i] * a.capacity + at[i];
        if (blockIdx.x == 0) a.offsets[x + rank[i]] = int32_t(min(at[i], a.capacity));
    }
    if (blockIdx.x == 0)
        for (uint32_t r = threadIdx.x; r < a.p; r += kSortThreads) {
            const uint32_t to = first_expert(a, r + 1);
            a.offsets[to + r] = int32_t(min(total_s[to] - total_s[first_expert(a, r)], a.capacity));
        }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4096 / kSortThreads; ++i) {
        const uint32_t x = threadIdx.x + i * kSortThreads;
        if (x < E) end_s[x] = (rank[i] + 1) * a.capacity;
    }
    __syncthreads();
    for (uint32_t g0 = begin; g0 < end; g0 += 32 * kSortItems) {
        if (!kept) {
            part.experts(g0 + lane, 32, e);
#pragma unroll
            for (int i = 0; i < kSortItems; ++i) {
                const int32_t *from = g0 + i * 32 + lane < end ? part.slot(g0 + i * 32 + lane) : nullptr;
                number[i] = from ? uint32_t(*from) : 0;
            }
        }
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const uint32_t g = g0 + i * 32 + lane;
            if (g >= end) break;
            uint32_t slot = ~0u;
            if (e[i] < E) {
                slot = begin_s[e[i]] + mine[e[i]] + number[i];      // (below 2^32)
                if (slot >= end_s[e[i]]) slot = ~0u;
            }
            if (int32_t *to = part.slot(g)) *to = int32_t(slot);
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
    const bool alone = a.all <= kSortAlone;
    // a part: a multiple of 32 choices; as many parts as SMs, or as the cells hold
    a.stride = (a.experts + 3) / 4 * 4;
    uint32_t parts = alone ? 1 : std::min<uint32_t>(std::min<uint32_t>(unsigned(L.num_sms), kSortCells / a.stride), (a.all + kSortPart - 1) / kSortPart);
    a.part = std::max<uint32_t>(1, uint32_t((uint64_t(a.all) + 32 * parts - 1) / (32 * parts))) * 32;
    a.parts = std::max<uint32_t>(1, (a.all + a.part - 1) / a.part);
    a.q = a.experts / a.p;
    a.rem = a.experts % a.p;
    a.warps = std::min<uint32_t>(kSortThreads / 32, kSortSmem / ((a.experts + 1) * 4));
    a.has_valid = N.valid ? 1 : 0;
    a.by_k = fast_div(a.k);
    a.by_rank = fast_div(a.per_rank ? a.per_rank : 1);
    a.by_q1 = fast_div(a.q + 1);
    a.by_q = fast_div(a.q ? a.q : 1);
    a.status = L.status;
    a.held = a.rows - (L.stall_test == 2 && a.rows ? 1 : 0);
    static std::atomic<unsigned long long> ready[6];
    const size_t smem = (size_t(a.experts) * 2 + 1 + size_t(a.warps) * (a.experts + 1)) * 4;
    const int bits = a.experts <= 16 ? 0 : a.experts <= 256 ? 1 : 2;
    void (*const places[6])(SortArgs<PM>) = {sort_place_kernel<PM, false, 4>, sort_place_kernel<PM, false, 8>, sort_place_kernel<PM, false, 12>,
                                             sort_place_kernel<PM, true, 4>,  sort_place_kernel<PM, true, 8>,  sort_place_kernel<PM, true, 12>};
    const int which = bits + (alone ? 3 : 0);
    void (*place)(SortArgs<PM>) = places[which];
    cudaError_t err = allow_dynamic_smem(place, kSortSmem + (2 * 4096 + 1) * 4, L.device, ready[which]);
    if (err != cudaSuccess) return err;
    info->kernel = "expert_sort";
    info->grid = int(a.parts);
    info->block = kSortThreads;
    info->smem = smem;
    if (!alone) {
        err = launch_dependent(sort_count_kernel<PM>, a.parts, kSortThreads, a.experts * 4, L.stream, a);
        if (err != cudaSuccess) return err;
        ++info->kernels;
    }
    err = launch_dependent(place, a.parts, kSortThreads, smem, L.stream, a);
    if (err == cudaSuccess) ++info->kernels;
    return err;
}

cudaError_t launch_expert_sort(const Launch &L, const SortLaunch &N, LaunchInfo *info)
{
    return L.p <= 8 ? sort_launch<8>(L, N, info) : sort_launch<kMaxRanks>(L, N, info);
}

}  // namespace ccl
