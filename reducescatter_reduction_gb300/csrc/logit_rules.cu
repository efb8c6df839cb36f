// Penalties for repeated tokens, biases and grammar masks on the logits of a
// decode step, the vocabulary split over the ranks.
//
// Per row, for token v, with c its occurrences among the generated tokens of
// the row's history, seen = it occurs anywhere in the history:
//   y = x + (sum of the row's bias entries for v)
//   y = y > 0 ? y / rep : y * rep      if seen
//   y = (y - freq * c) - pres          if c > 0
//   y = -inf                           if the row's mask has bit v clear
// in fp32, rounded once to the element type.
//
// One CTA per (row, rank, slice of the rank's columns).  It starts the copies
// of its groups into shared memory, all but those that the row's mask forbids
// altogether, and meanwhile counts the row's history: the tokens that fall
// into the slice, in one counter per column in shared memory (integer
// atomics, so any order gives the same counts); who raises a counter from
// zero puts its column on a list.  Each warp queues the tokens that it finds,
// so that the counting runs with full warps.  The row's bias entries for the
// slice are kept in their order, and their columns go on the list too.  Then
// the listed columns are done in shared memory, each by a lane of its own (in
// the groups' own lanes the rules cost more than the copy: a history of
// thousands of tokens touches few columns, but nearly every group of 32 lanes
// has one), and the groups go out through their mask bits.  Where every rank
// is in place nothing is staged: only groups that the mask changes are read
// and written, and the listed columns in memory.  Counters are 16 bits wide
// where the history is shorter than 2^14 tokens.  Bytes: the logits once in
// and once out, the history once per slice (L2).  Bound by launch and latency
// where there are few (1 x 32000 f32: 4.5 us), else by the counting of the
// history: 512 x 131072 bf16 take 100 us (2.8 TB/s) with histories of up to
// 8192 tokens, 48 without, of which copy and mask alone are 45 (6.1 TB/s).
#include "async.cuh"
#include "logits.cuh"

namespace ccl {

template <int PM>
struct RulesArgs {
    Shards<PM> s;
    ccl_logit_rules_t r;
    uint32_t slices;            // per rank
    FastDiv by_row, by_slices;  // CTAs per row, slices per rank
    int in_place;               // every rank's output is its input
};

// A column's counter: bit 0 says "in the prompt", the top bit "has a bias
// entry", and generated occurrences are counted between them.
constexpr uint32_t kSeenPrompt = 1, kGenerated = 2;
// Bias entries of a slice that are kept in shared memory, where each column
// that has one goes through them; with more, whole blocks of columns are
// summed in walks through the row's list.
constexpr uint32_t kBiasKept = 256;

// Clears the lanes of a group that the mask bits forbid to -inf.
template <typename T>
__device__ __forceinline__ uint4 forbid(const uint4 &v, uint32_t allowed)
{
    const uint32_t low = lowest_group<T>().x;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (Traits<T>::VEC == 4) {
            w[i] = (allowed >> i) & 1 ? w[i] : low;
        } else {
            const uint32_t keep = ((allowed >> (2 * i)) & 1 ? 0xffffu : 0u) | ((allowed >> (2 * i + 1)) & 1 ? 0xffff0000u : 0u);
            w[i] = (w[i] & keep) | (low & ~keep);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int PM, int THREADS, int NV, bool WIDE>
__global__ void __launch_bounds__(THREADS, THREADS > 256 ? 2 : 3) logit_rules_kernel(const __grid_constant__ RulesArgs<PM> a)
{
    using Tr = Traits<T>;
    constexpr int VEC = Tr::VEC, GROUPS = THREADS * NV, PER = WIDE ? 1 : 2;   // counters per word
    constexpr int CELLS = (GROUPS + 2) * VEC;       // a group's room before and after for the edges
    constexpr uint32_t BITS = 32 / PER, BIASED = 1u << (BITS - 1), ONES = BIASED | (BIASED - 1);
    constexpr uint32_t LIST = CELLS < 2048 ? CELLS : 2048;   // columns the list holds; with more, it is made anew for as many counters
    constexpr int WARPS = THREADS / 32, BATCH = THREADS > 256 ? 4 : 8;   // tokens a thread loads at once
    extern __shared__ uint4 smem4[];
    uint4 *stage = smem4;                            // the slice's logits, a cell an element
    uint32_t *cnt = reinterpret_cast<uint32_t *>(smem4 + (a.in_place ? 0 : CELLS / VEC));
    struct Scan {
        uint16_t queue[WARPS][32 * (BATCH + 1)];    // tokens found: cell, and whether generated in the top bit
        uint16_t list[LIST];
    };
    __shared__ __align__(16) Scan scan;
    constexpr uint32_t SUMS = 2048, PART = SUMS / WARPS;    // columns whose biases are summed at once, a warp's part of them
    static_assert(sizeof(Scan) >= SUMS * sizeof(float), "the sums have the room of the queues and the list");
    uint16_t *list = scan.list;
    __shared__ uint16_t bias_cell[kBiasKept];
    __shared__ float bias_value[kBiasKept];
    __shared__ uint32_t bias_found[WARPS];
    __shared__ uint32_t listed;
    const Shards<PM> &s = a.s;
    const uint32_t row32 = div_by(blockIdx.x, a.by_row), rest = blockIdx.x - row32 * a.by_row.d;
    const uint32_t rank = div_by(rest, a.by_slices), slice = rest - rank * a.slices;
    const uint64_t row = row32;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const ShardRow<T, PM> in(s, s.in[rank], rank, row);
    const uint32_t whole = in.end - in.first;
    if (slice > 0 && slice * GROUPS >= whole) return;
    const uint32_t j0 = in.first + slice * GROUPS, j1 = min(j0 + GROUPS, in.end);
    const bool has_tail = j1 == in.end;
    // the slice's columns are [c0, c1); column c has cell c - cell0
    const uint32_t c0 = slice == 0 ? 0 : in.head() + slice * GROUPS * VEC, c1 = has_tail ? in.width : in.head() + (j1 - in.first) * VEC;
    const int cell0 = int(in.head() + slice * GROUPS * VEC) - VEC;
    const uint32_t token0 = shard_begin(s, rank), from = token0 + c0, width = c1 - c0;
    const uint32_t cell_from = uint32_t(int(c0) - cell0);
    const int edge = in.edge(tid, slice == 0, has_tail);

    const bool history = a.r.history != nullptr;
    if (tid == 0) listed = 0;
    if (history || a.r.bias_count)
        for (int i = tid; i < CELLS / PER / 4; i += THREADS) reinterpret_cast<uint4 *>(cnt)[i] = make_uint4(0, 0, 0, 0);
    grid_dependency_wait();
    grid_dependents_launch();

    // the row's rules, all loads at once, and the first tokens of its history whether they count or not
    const bool listed_row = row_held(s, row);      // (checked build: the lists have this row)
    const int mask_at = a.r.mask && a.r.mask_index ? (listed_row ? a.r.mask_index[row] : -1) : int(row);
    const int ld = history && listed_row ? int(a.r.history_ld) : 0;
    const int32_t *h = history ? a.r.history + row * a.r.history_ld : nullptr;
    int len = ld && a.r.history_len ? a.r.history_len[row] : ld;
    const int prompt = ld && a.r.prompt_len ? a.r.prompt_len[row] : 0;
    const bool lists = a.r.bias_count && listed_row;
    const int offset0 = lists ? a.r.bias_offsets[row] : 0, offset1 = lists ? a.r.bias_offsets[row + 1] : 0;
    auto held_token = [&](int j) { return in_bounds(uint64_t(row) * a.r.history_ld + j < s.held * a.r.history_ld, s.status, s.site, j); };
    int32_t token[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) token[k] = tid + k * THREADS < ld && held_token(tid + k * THREADS) ? h[tid + k * THREADS] : -1;

    // the mask bits of this thread's groups, then the logits of those that have any
    const uint32_t *mask = a.r.mask && mask_at >= 0 && uint64_t(mask_at) < a.r.mask_rows ? a.r.mask + uint64_t(mask_at) * a.r.mask_ld : nullptr;
    constexpr uint32_t ALL = (1u << VEC) - 1;
    constexpr int PACK = 32 / VEC, MASKS = (NV + PACK - 1) / PACK;      // groups whose bits a word holds
    uint32_t allowed[MASKS];
#pragma unroll
    for (int i = 0; i < MASKS; ++i) allowed[i] = 0xffffffffu;
    const uint32_t words = (s.vocab + 31) / 32;
    auto word_of = [&](uint32_t w) -> uint32_t {
        return in_bounds(uint64_t(mask_at) < a.r.mask_rows && w < words, s.status, s.site, w) ? mask[w] : 0u;
    };
    auto ok_of = [&](int n) -> uint32_t { return (allowed[n / PACK] >> (n % PACK * VEC)) & ALL; };
    if (mask) {
        const uint32_t v0 = token0 + (j0 + tid) * VEC - in.shift;
        uint32_t lo[NV], hi[NV];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const uint32_t w = (v0 + n * THREADS * VEC) >> 5;
            const bool is = j0 + tid + n * THREADS < j1;
            lo[n] = is ? word_of(w) : 0u;
            hi[n] = is && w + 1 < words ? word_of(w + 1) : 0u;
        }
#pragma unroll
        for (int i = 0; i < MASKS; ++i) allowed[i] = 0;
#pragma unroll
        for (int n = 0; n < NV; ++n)
            allowed[n / PACK] |= (__funnelshift_r(lo[n], hi[n], (v0 + n * THREADS * VEC) & 31) & ALL) << (n % PACK * VEC);
    }
    if (!a.in_place) {
        const uint32_t to = smem_addr(stage) + (tid + 1) * 16;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const uint32_t j = j0 + tid + n * THREADS;
            if (j < j1 && ok_of(n) && in.holds_group(j))
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + n * THREADS * 16), "l"(in.group(j)) : "memory");
        }
        if (edge >= 0) Tr::store1(stage, uint64_t(edge - cell0), in.column(edge));
    }
    // the row's entries [bias_lo, bias_hi), held to the list; unsigned, as a block that begins below 2^31 may end beyond
    const uint32_t bias_lo = min(uint32_t(max(offset0, 0)), uint32_t(a.r.bias_count));
    const uint32_t bias_hi = max(bias_lo, min(uint32_t(max(offset1, 0)), uint32_t(a.r.bias_count)));
    len = len < 0 ? 0 : len > ld ? ld : len;
    uint32_t bias_token = 0xffffffffu;     // of this thread's entry in a block of the list, from the slice's first
    float bias_add = 0.0f;
    auto held_entry = [&](uint32_t k) { return in_bounds(k < a.r.bias_count, s.status, s.site, k); };
    auto entry = [&](uint32_t k) {
        const bool is = k < bias_hi && held_entry(k);
        bias_token = is ? uint32_t(a.r.bias_tokens[k]) - from : 0xffffffffu;
        bias_add = is ? a.r.bias_values[k] : 0.0f;
    };
    entry(bias_lo + tid);
    __syncthreads();

    // A whole warp raises the counters of its lanes' cells (where `is`); who raises one from zero lists it.
    auto raise = [&](bool is, uint32_t cell, uint32_t what, bool by_or) {
        const uint32_t sh = WIDE ? 0 : (cell % 2) * 16;
        uint32_t old = ONES << sh;
        if (is) old = by_or ? atomicOr(&cnt[cell / PER], what << sh) : atomicAdd(&cnt[cell / PER], what << sh);
        const bool fresh = is && ((old >> sh) & ONES) == 0;
        const unsigned who = __ballot_sync(0xffffffffu, fresh);
        if (!who) return;
        uint32_t at = 0;
        if (lane == __ffs(who) - 1) at = atomicAdd(&listed, uint32_t(__popc(who)));
        at = __shfl_sync(0xffffffffu, at, __ffs(who) - 1) + __popc(who & ((1u << lane) - 1));
        if (fresh && at < LIST) list[at] = uint16_t(cell);
    };
    uint16_t *q = scan.queue[warp];
    int queued = 0;
#pragma unroll 1
    for (int j = tid; j - lane < len; j += BATCH * THREADS) {
        if (j != tid) {
#pragma unroll
            for (int k = 0; k < BATCH; ++k) token[k] = j + k * THREADS < len && held_token(j + k * THREADS) ? h[j + k * THREADS] : -1;
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const uint32_t c = uint32_t(token[k]) - from;        // another slice's, or no token: not below width
            const int at = j + k * THREADS;
            const bool is = c < width && at < len;
            const unsigned who = __ballot_sync(0xffffffffu, is);
            if (is) q[queued + __popc(who & ((1u << lane) - 1))] = uint16_t((c + cell_from) | (at < prompt ? 0u : 0x8000u));
            queued += __popc(who);
        }
        __syncwarp();
        // whole warps of the queue; the rest stays for the next batch, or is done with the last
        const bool more = j - lane + BATCH * THREADS < len;
        int done = 0;
#pragma unroll 1
        for (; done + (more ? 32 : 1) <= queued; done += 32) {
            const bool is = done + lane < queued;
            const uint32_t e = is ? q[done + lane] : 0u, made = e >> 15;
            raise(is, e & 0x7fff, made ? kGenerated : kSeenPrompt, !made);
        }
        if (more) {
            const uint16_t rest = done + lane < queued ? q[done + lane] : uint16_t(0);
            __syncwarp();
            queued -= done;
            if (lane < queued) q[lane] = rest;
        }
    }
    uint32_t kept = 0;
    for (uint32_t b = bias_lo; b < bias_hi; b += THREADS) {
        // the list's entries for the slice, in their order
        if (b > bias_lo) entry(b + tid);
        const bool is = b + tid < bias_hi && bias_token < width;
        const unsigned who = __ballot_sync(0xffffffffu, is);
        if (lane == 0) bias_found[warp] = __popc(who);
        __syncthreads();
        uint32_t before = kept;
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) before += bias_found[w];
            kept += bias_found[w];
        }
        if (who) {
            const uint32_t at = before + __popc(who & ((1u << lane) - 1));
            if (is && at < kBiasKept) {
                bias_cell[at] = uint16_t(bias_token + cell_from);
                bias_value[at] = bias_add;
            }
            raise(is, bias_token + cell_from, BIASED, true);
        }
        if (b + THREADS < bias_hi) __syncthreads();
    }

    const ShardRow<T, PM> out(s, s.out[rank], rank, row);
    auto may = [&](uint32_t col) { return !mask || (word_of((token0 + col) >> 5) >> ((token0 + col) & 31)) & 1; };
    if (a.in_place) {
        // what the mask forbids
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const uint32_t j = j0 + tid + n * THREADS, ok = ok_of(n);
            if (j < j1 && ok != ALL) store_group<T>(out, in, j, forbid<T>(ok && in.holds_group(j) ? ld_coherent_v4(in.group(j)) : lowest_group<T>(), ok));
        }
        if (edge >= 0 && !may(edge)) out.set_column(edge, -INFINITY);
    } else {
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __syncthreads();

    // the listed columns: in shared memory, or in place where they are allowed
    const float rep = a.r.repetition && listed_row ? a.r.repetition[row] : 1.0f;
    const float freq = a.r.frequency && listed_row ? a.r.frequency[row] : 0.0f;
    const float pres = a.r.presence && listed_row ? a.r.presence[row] : 0.0f;
    auto counter = [&](uint32_t cell) -> uint32_t { return (cnt[cell / PER] >> (WIDE ? 0 : (cell % 2) * 16)) & ONES; };
    auto changed = [&](float y, uint32_t c, float bias) -> float {
        if (c & BIASED) y = __fadd_rn(y, bias);
        const uint32_t seen = c & (BIASED - 1);
        if (seen) y = y > 0.0f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
        if (seen >= kGenerated) y = __fsub_rn(__fsub_rn(y, __fmul_rn(freq, float(seen >> 1))), pres);
        return y;
    };
    if (kept > kBiasKept) {
        // More entries than are kept: the sums of SUMS columns at a time, a part of them by each warp, which walks through
        // all of the row's entries in their order.  So the time goes with the list's length: 64 x 32000 bf16 with 3200
        // entries a row 114 us, with 32000 895 (214 and 26700 where each column went through the list by itself).
        float *sums = reinterpret_cast<float *>(&scan);
        for (uint32_t first = 0; first < width; first += SUMS) {
            __syncthreads();
            float *mine = sums + warp * PART;
            for (uint32_t i = lane; i < PART; i += 32) mine[i] = 0.0f;
            __syncwarp();
            const uint32_t part = from + first + warp * PART;
            constexpr int M = 4;          // loads in flight
#pragma unroll 1
            for (uint32_t b = bias_lo + lane; b - lane < bias_hi; b += 32 * M) {
                uint32_t at[M];
                float v[M];
#pragma unroll
                for (int k = 0; k < M; ++k) {
                    const bool in = b + 32 * k < bias_hi && held_entry(b + 32 * k);
                    at[k] = in ? uint32_t(a.r.bias_tokens[b + 32 * k]) - part : 0xffffffffu;
                    v[k] = in ? a.r.bias_values[b + 32 * k] : 0.0f;
                }
#pragma unroll
                for (int k = 0; k < M; ++k) {
                    const bool is = at[k] < PART;
                    if (!__any_sync(0xffffffffu, is)) continue;
                    // a column's entries one after the other, by the lanes before that have it too
                    const unsigned same = __match_any_sync(0xffffffffu, is ? at[k] : 0x80000000u | uint32_t(lane));
                    const int turn = __popc(same & ((1u << lane) - 1));
                    for (int t = 0; __any_sync(0xffffffffu, is && turn >= t); ++t) {
                        if (is && turn == t) mine[at[k]] = __fadd_rn(mine[at[k]], v[k]);
                        __syncwarp();
                    }
                }
            }
            __syncthreads();
            for (uint32_t i = tid; i < min(SUMS, width - first); i += THREADS) {
                const uint32_t cell = first + i + cell_from, col = cell + uint32_t(cell0), c = counter(cell);
                if (!c || (a.in_place && !may(col))) continue;
                const float y = changed(a.in_place ? in.column(col) : Tr::load1(stage, cell), c, sums[i]);
                if (a.in_place) out.set_column(col, y);
                else Tr::store1(stage, cell, y);
            }
        }
    } else {
        const bool fits = listed <= LIST;
        for (uint32_t first = 0; first < (fits ? 1u : width); first += LIST) {
            if (!fits) {
                // the next LIST counters' columns
                __syncthreads();
                if (tid == 0) listed = 0;
                __syncthreads();
                for (uint32_t c = first + tid; c < min(first + LIST, width); c += THREADS)
                    if (counter(c + cell_from)) list[atomicAdd(&listed, 1u)] = uint16_t(c + cell_from);
                __syncthreads();
            }
            const uint32_t count = listed;
            constexpr int AT_ONCE = 2;
#pragma unroll 1
            for (uint32_t i = tid; i < count; i += AT_ONCE * THREADS) {
                uint32_t cell[AT_ONCE], bits = 0;
                float x[AT_ONCE];
#pragma unroll
                for (int k = 0; k < AT_ONCE; ++k) {
                    const bool is = i + k * THREADS < count;
                    cell[k] = is ? list[i + k * THREADS] : cell_from;
                    x[k] = 0.0f;
                    if (is) {
                        const uint32_t col = cell[k] + uint32_t(cell0);
                        x[k] = a.in_place ? in.column(col) : Tr::load1(stage, cell[k]);
                        bits |= (!a.in_place || may(col) ? 1u : 0u) << k;
                    }
                }
#pragma unroll
                for (int k = 0; k < AT_ONCE; ++k) {
                    if (!((bits >> k) & 1)) continue;
                    const uint32_t c = counter(cell[k]);
                    float sum = 0.0f;
                    if (c & BIASED)
                        for (uint32_t b = 0; b < kept; ++b)
                            if (bias_cell[b] == cell[k]) sum = __fadd_rn(sum, bias_value[b]);
                    const float y = changed(x[k], c, sum);
                    if (a.in_place) out.set_column(cell[k] + uint32_t(cell0), y);
                    else Tr::store1(stage, cell[k], y);
                }
            }
        }
    }
    if (a.in_place) return;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const uint32_t j = j0 + tid + n * THREADS, ok = ok_of(n);
        if (j >= j1) break;
        store_group<T>(out, in, j, ok == ALL ? stage[tid + n * THREADS + 1] : ok ? forbid<T>(stage[tid + n * THREADS + 1], ok) : lowest_group<T>());
    }
    if (edge >= 0) out.set_column(edge, may(edge) ? Tr::load1(stage, uint64_t(edge - cell0)) : -INFINITY);
}

template <typename T, int PM, int THREADS, int NV, bool WIDE>
static cudaError_t rules_launch(const Launch &L, RulesArgs<PM> &a, uint32_t groups, LaunchInfo *info)
{
    constexpr uint32_t GROUPS = THREADS * NV;
    constexpr size_t counters = size_t(GROUPS + 2) * Traits<T>::VEC * (WIDE ? 4 : 2), staged = size_t(GROUPS + 2) * 16;
    const size_t smem = counters + (a.in_place ? 0 : staged);
    a.slices = groups ? (groups + GROUPS - 1) / GROUPS : 1;
    const uint64_t per_row = uint64_t(a.slices) * a.s.p;
    if (a.s.rows * per_row > 0x7fffffffull) return kTooManyPieces;
    a.by_row = fast_div(uint32_t(per_row));
    a.by_slices = fast_div(a.slices);
    static std::atomic<unsigned long long> done{0};
    cudaError_t err = allow_dynamic_smem(logit_rules_kernel<T, PM, THREADS, NV, WIDE>, counters + staged, L.device, done);
    if (err != cudaSuccess) return err;
    const unsigned grid = unsigned(a.s.rows * per_row);
    err = launch_dependent(logit_rules_kernel<T, PM, THREADS, NV, WIDE>, grid, THREADS, smem, L.stream, a);
    if (err != cudaSuccess) return err;
    info->kernel = "logit_rules";
    info->grid = int(grid);
    info->block = THREADS;
    info->smem = smem;
    info->kernels = 1;
    return cudaGetLastError();
}

template <typename T, int PM, bool WIDE>
static cudaError_t rules_shape(const Launch &L, const RulesLaunch &N, LaunchInfo *info)
{
    constexpr int PER16 = Traits<T>::VEC == 8 ? 1 : 2;   // groups that hold eight elements
    RulesArgs<PM> a;
    fill_shards(&a.s, L, N.rows, N.vocab, N.ld, kSiteRules);
    a.r = *N.rules;
    a.in_place = L.alias ? 1 : 0;
    const uint32_t groups = widest_groups<T>(a.s);
    const uint64_t all = N.rows * a.s.p * uint64_t(groups), sms = uint64_t(L.num_sms);
    // Few logits: small slices and many threads to go through the history at
    // once; many: large slices, as each goes through the history again.
    // Measured (graph replay, us; 512 x PER16, 512 x 4, 256 x 8 threads x
    // groups): 1 x 32000 f32, history 2048: 4.5, 5.2, 6.0; 48 x 50021 f16,
    // history 4000: 15.8, 10.4, 13.2; 512 x 131072 bf16, history up to 8192:
    // 286, 118, 100, and next to none: 178, 65, 48.
    if (all < sms * 1024 * PER16) return rules_launch<T, PM, 512, PER16, WIDE>(L, a, groups, info);
    if (all < sms * 4096 * PER16) return rules_launch<T, PM, 512, 4, WIDE>(L, a, groups, info);
    return rules_launch<T, PM, 256, 8, WIDE>(L, a, groups, info);
}

template <typename T>
static cudaError_t rules_dtype(const Launch &L, const RulesLaunch &N, LaunchInfo *info)
{
    // a 16-bit counter holds twice the occurrences, plus one, below its top bit
    const bool wide = N.rules->history && N.rules->history_ld > 16383;
    if (wide) return L.p <= 8 ? rules_shape<T, 8, true>(L, N, info) : rules_shape<T, kMaxRanks, true>(L, N, info);
    return L.p <= 8 ? rules_shape<T, 8, false>(L, N, info) : rules_shape<T, kMaxRanks, false>(L, N, info);
}

cudaError_t launch_logit_rules(const Launch &L, const RulesLaunch &N, LaunchInfo *info)
{
    switch (L.dtype) {
    case DT_F32: return rules_dtype<F32>(L, N, info);
    case DT_F16: return rules_dtype<F16>(L, N, info);
    case DT_BF16: return rules_dtype<BF16>(L, N, info);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace ccl
