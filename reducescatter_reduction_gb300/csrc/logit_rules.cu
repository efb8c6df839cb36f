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
// One CTA per (row, rank, slice of the rank's columns).  It starts the loads
// of the row's rules, of the first part of its history and of its own groups,
// then counts the history's tokens that fall into the slice in one counter
// per column in shared memory (integer atomics, so any order gives the same
// counts), adds up the row's bias entries in list order (one warp), and
// finishes its groups: one that neither touches is copied through its mask
// bits as it is.  A group that its mask forbids altogether is not read, and in
// place an untouched one is not written.  Counters are 16 bits wide where the
// history is shorter than 2^15 tokens: half the shared memory to clear and to
// read.  Bytes: the logits once in and once out, plus the history once per
// slice (L2).
#include "logits.cuh"

namespace ccl {

template <int PM>
struct RulesArgs {
    Shards<PM> s;
    ccl_logit_rules_t r;
    uint32_t slices;            // per rank
    uint32_t cluster;           // CTAs that share the scan of a row's history
    FastDiv by_row, by_slices;  // CTAs per row (whole clusters), slices per rank
    int in_place;
};

// From this many tokens on, the CTAs of a cluster share the scan of a row's
// history; below, each scans it all and saves the cluster's barriers.
constexpr size_t kShareHistory = 1024;
constexpr uint32_t kScanCluster = 8;

// Generated occurrences sit above bit 0, bit 0 says "in the prompt".
constexpr uint32_t kSeenPrompt = 1, kGenerated = 2;

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
__global__ void __launch_bounds__(THREADS) logit_rules_kernel(const __grid_constant__ RulesArgs<PM> a)
{
    using Tr = Traits<T>;
    constexpr int VEC = Tr::VEC, GROUPS = THREADS * NV, PER = WIDE ? 1 : 2;   // counters per word
    constexpr int CELLS = (GROUPS + 2) * VEC;       // a group's room before and after for the edges
    static_assert(NV * VEC <= 32, "the mask bits of a thread fit one word");
    extern __shared__ uint4 smem4[];
    uint32_t *cnt = reinterpret_cast<uint32_t *>(smem4);
    float *bias = reinterpret_cast<float *>(cnt + CELLS / PER);
    __shared__ uint32_t biased_groups[GROUPS / 32];       // bit g: group g has a bias entry
    __shared__ uint32_t list_cell[THREADS], list_count[THREADS / 32];
    __shared__ float list_value[THREADS];
    __shared__ uint32_t head_s[PM], last_s[PM];           // a rank's head, its last slice (shared scan)
    const Shards<PM> &s = a.s;
    const uint32_t row32 = div_by(blockIdx.x, a.by_row), mine = blockIdx.x - row32 * a.by_row.d;
    const uint32_t rank_of_mine = div_by(mine, a.by_slices), slice = mine - rank_of_mine * a.slices;
    const uint64_t row = row32;
    const int tid = threadIdx.x;
    const bool shared_scan = a.cluster > 1;
    bool here = rank_of_mine < s.p;                       // else: only in the scan
    const uint32_t rank = here ? rank_of_mine : 0;
    const ShardRow<T> in(s.in[rank], s.ld, row, shard_width(s, rank));
    const uint32_t whole = in.end - in.first;
    here = here && (slice == 0 || slice * GROUPS < whole) && in_bounds(row < s.rows, s.status, kSiteRules, row);
    if (!here && !shared_scan) return;
    const uint32_t j0 = in.first + min(slice * GROUPS, whole), j1 = here ? min(j0 + GROUPS, in.end) : j0;
    const bool has_tail = here && j1 == in.end;
    // the slice's columns are [c0, c1); column c has cell c - cell0
    const uint32_t c0 = slice == 0 ? 0 : in.head() + slice * GROUPS * VEC, c1 = !here ? c0 : has_tail ? in.width : in.head() + (j1 - in.first) * VEC;
    const int cell0 = int(in.head() + slice * GROUPS * VEC) - VEC;
    const uint32_t token0 = shard_begin(s, rank);
    const int edge = here ? in.edge(tid, slice == 0, has_tail) : -1;

    const bool history = a.r.history != nullptr;
    if (tid < GROUPS / 32) biased_groups[tid] = 0;
    if (history)
        for (int i = tid; i < CELLS / PER / 4; i += THREADS) reinterpret_cast<uint4 *>(cnt)[i] = make_uint4(0, 0, 0, 0);
    if (shared_scan) {
        if (tid < int(s.p)) {
            const ShardRow<T> sr(s.in[tid], s.ld, row, shard_width(s, tid));
            head_s[tid] = sr.head();
            last_s[tid] = sr.end > sr.first ? (sr.end - sr.first - 1) / GROUPS : 0;
        }
        // every counter of the cluster is zero before anyone counts
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    grid_dependency_wait();
    grid_dependents_launch();

    // the row's rules, all loads at once, and the first tokens of its history whether they count or not
    const int mask_at = a.r.mask && a.r.mask_index ? a.r.mask_index[row] : int(row);
    constexpr int BATCH = THREADS <= 128 ? 8 : 4;
    const uint32_t scan_rank = shared_scan ? mine % a.cluster : 0, scan_step = THREADS * a.cluster;
    const int scan0 = int(scan_rank) * THREADS + tid;
    const int ld = history ? int(a.r.history_ld) : 0;
    const int32_t *h = a.r.history + row * a.r.history_ld;
    int len = history && a.r.history_len ? a.r.history_len[row] : ld;
    const int prompt = history && a.r.prompt_len ? a.r.prompt_len[row] : 0;
    int bias_lo = a.r.bias_count ? a.r.bias_offsets[row] : 0, bias_hi = a.r.bias_count ? a.r.bias_offsets[row + 1] : 0;
    const float rep = a.r.repetition ? a.r.repetition[row] : 1.0f;
    const float freq = a.r.frequency ? a.r.frequency[row] : 0.0f;
    const float pres = a.r.presence ? a.r.presence[row] : 0.0f;
    int32_t token[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) token[k] = scan0 + k * scan_step < ld ? h[scan0 + k * scan_step] : -1;

    // the mask bits of this thread's groups, VEC for each, then the logits of those that have any
    const uint32_t *mask = a.r.mask && mask_at >= 0 && uint64_t(mask_at) < a.r.mask_rows ? a.r.mask + uint64_t(mask_at) * a.r.mask_ld : nullptr;
    constexpr uint32_t ALL = (1u << VEC) - 1;
    uint32_t allowed = 0xffffffffu;
    if (mask) {
        const uint32_t words = (s.vocab + 31) / 32;
        const uint32_t v0 = token0 + (j0 + tid) * VEC - in.shift;
        uint32_t lo[NV], hi[NV];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const uint32_t w = (v0 + n * THREADS * VEC) >> 5;
            const bool is = j0 + tid + n * THREADS < j1;
            lo[n] = is ? mask[w] : 0u;
            hi[n] = is && w + 1 < words ? mask[w + 1] : 0u;
        }
        allowed = 0;
#pragma unroll
        for (int n = 0; n < NV; ++n) allowed |= (__funnelshift_r(lo[n], hi[n], (v0 + n * THREADS * VEC) & 31) & ALL) << (n * VEC);
    }
    uint4 raw[NV];
    auto fetch = [&]() {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const uint32_t j = j0 + tid + n * THREADS;
            if (j < j1 && (allowed >> (n * VEC)) & ALL) raw[n] = ld_coherent_v4(in.group(j));
            else raw[n] = lowest_group<T>();
        }
    };
    if (!a.in_place) fetch();
    const float edge_x = edge >= 0 ? in.column(edge) : 0.0f;

    if (a.r.bias_count) {
        const int n = int(a.r.bias_count);
        bias_lo = bias_lo < 0 ? 0 : bias_lo > n ? n : bias_lo;
        bias_hi = bias_hi < bias_lo ? bias_lo : bias_hi > n ? n : bias_hi;
    }
    const bool biased = here && bias_hi > bias_lo;
    len = len < 0 ? 0 : len > ld ? ld : len;
    uint32_t bias_col = 0xffffffffu;      // this thread's entry of the first THREADS
    float bias_add = 0.0f;
    if (biased && bias_lo + tid < bias_hi) {
        bias_col = uint32_t(a.r.bias_tokens[bias_lo + tid]) - token0;
        bias_add = a.r.bias_values[bias_lo + tid];
    }
    __syncwarp();
    if (shared_scan) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    else __syncthreads();
    if (len) {
        auto count_at = [&](uint32_t at, int cell, int j) {
            // cell's counter in the shared memory at `at` (a cluster address)
            const uint32_t word = at + uint32_t(WIDE ? cell : cell / 2) * 4, sh = WIDE ? 0 : (cell % 2) * 16;
            if (j < prompt) asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(word), "r"(kSeenPrompt << sh) : "memory");
            else asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(word), "r"(kGenerated << sh) : "memory");
        };
        const uint32_t cnt_at = uint32_t(__cvta_generic_to_shared(cnt));
        auto count = [&](uint32_t v, int j) {
            if (j >= len) return;
            if (!shared_scan) {
                const uint32_t c = v - token0;
                if (c - c0 < c1 - c0) count_at(cnt_at, int(c) - cell0, j);   // else another slice's, or no token
                return;
            }
            if (v >= s.vocab) return;
            const uint32_t r = rank_of_token(s, v), c = v - shard_begin(s, r), head = head_s[r];
            const uint32_t sl = c < head ? 0u : min((c - head) / (GROUPS * VEC), last_s[r]);
            const uint32_t to = r * a.slices + sl - (mine - scan_rank);
            if (to >= a.cluster) return;                                     // another cluster's
            uint32_t at;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(cnt_at), "r"(to));
            count_at(at, int(c) - int(head + sl * GROUPS * VEC) + VEC, j);
        };
#pragma unroll
        for (int k = 0; k < BATCH; ++k) count(uint32_t(token[k]), scan0 + k * scan_step);
        for (int j = scan0 + BATCH * scan_step; j < len; j += BATCH * scan_step) {
#pragma unroll
            for (int k = 0; k < BATCH; ++k) token[k] = j + k * scan_step < uint32_t(len) ? h[j + k * scan_step] : -1;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) count(uint32_t(token[k]), j + k * scan_step);
        }
    }
    __syncwarp();
    if (shared_scan) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (biased) {
        // The sums of the edges begin at zero, those of a group when its first entry comes.
        const int tail = VEC + int(j1 - j0) * VEC, lane = tid % 32;
        if (tid < VEC) bias[tid] = 0.0f;
        else if (tid < 2 * VEC) bias[tail + tid - VEC] = 0.0f;
        for (int b = bias_lo; b < bias_hi; b += THREADS) {
            // a block of entries: each warp lists those of the slice in order ...
            if (b > bias_lo) {
                const bool is = b + tid < bias_hi;
                bias_col = is ? uint32_t(a.r.bias_tokens[b + tid]) - token0 : 0xffffffffu;
                bias_add = is ? a.r.bias_values[b + tid] : 0.0f;
                __syncthreads();      // the last block's list is done with
            }
            const bool in_slice = b + tid < bias_hi && bias_col - c0 < c1 - c0;
            const unsigned who = __ballot_sync(0xffffffffu, in_slice);
            if (lane == 0) list_count[tid / 32] = __popc(who);
            if (in_slice) {
                const int cell = int(bias_col) - cell0, g = cell / VEC - 1, at = tid - lane + __popc(who & ((1u << lane) - 1));
                list_cell[at] = uint32_t(cell);
                list_value[at] = bias_add;
                if (g >= 0 && g < int(j1 - j0) && !((atomicOr(&biased_groups[g / 32], 1u << (g % 32)) >> (g % 32)) & 1)) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) bias[(g + 1) * VEC + i] = 0.0f;
                }
            }
            __syncthreads();
            // ... and the last warp adds the lists up, entries of one token in list order
            if (tid < THREADS - 32) continue;
            for (int w = 0; w < THREADS / 32; ++w) {
                const int n = int(list_count[w]);
                if (n == 0) continue;
                const uint32_t cell = lane < n ? list_cell[32 * w + lane] : 0xffffffffu;
                const float add = lane < n ? list_value[32 * w + lane] : 0.0f;
                const unsigned same = __match_any_sync(0xffffffffu, cell);
                const int turn = lane < n ? __popc(same & ((1u << lane) - 1)) : -1;
                for (int t = 0; __any_sync(0xffffffffu, turn >= t); ++t) {
                    if (turn == t) bias[cell] = __fadd_rn(bias[cell], add);
                    __syncwarp();
                }
            }
        }
    }
    __syncwarp();
    if (shared_scan) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    __syncthreads();
    if (!here) return;

    auto apply = [&](float x, uint32_t c, float b) -> float {
        if (b != 0.0f) x = __fadd_rn(x, b);
        if (c) x = x > 0.0f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
        if (c >= kGenerated) x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, float(c >> 1))), pres);
        return x;
    };
    const ShardRow<T> out(s.out[rank], s.ld, row, in.width);
    if (a.in_place) fetch();
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int g = tid + n * THREADS;
        const uint32_t j = j0 + g, ok = (allowed >> (n * VEC)) & ALL;
        if (j >= j1) break;
        uint4 v = raw[n];
        bool changed = ok != ALL;
        if (ok) {
            constexpr int WORDS = VEC / PER;
            uint32_t c[WORDS], any = 0;
            if (len) {
                const uint32_t *at = cnt + (g + 1) * WORDS;
#pragma unroll
                for (int i = 0; i < WORDS; ++i) {
                    c[i] = at[i];
                    any |= c[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < WORDS; ++i) c[i] = 0;
            }
            const bool sums = biased && (biased_groups[g / 32] >> (g % 32)) & 1;
            if (any || sums) {
                float x[VEC];
                Tr::unpack(v, x);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    x[i] = apply(x[i], WIDE ? c[i] : (c[i / PER] >> (16 * (i % PER))) & 0xffffu, sums ? bias[(g + 1) * VEC + i] : 0.0f);
                v = Tr::pack(x);
                changed = true;
            }
        }
        if (a.in_place && !changed) continue;
        if (ok != ALL) v = forbid<T>(v, ok);
        store_group<T>(out, in, j, v);
    }
    if (edge >= 0) {
        const uint32_t v = token0 + edge;
        const bool ok = !mask || (mask[v >> 5] >> (v & 31)) & 1;
        const int cell = edge - cell0;
        const uint32_t c = !len ? 0u : WIDE ? cnt[cell] : (cnt[cell / 2] >> (16 * (cell % 2))) & 0xffffu;
        out.set_column(edge, ok ? apply(edge_x, c, biased ? bias[cell] : 0.0f) : -INFINITY);
    }
}

template <typename T, int PM, int THREADS, int NV, bool WIDE>
static cudaError_t rules_launch(const Launch &L, RulesArgs<PM> &a, uint32_t groups, bool share, LaunchInfo *info)
{
    constexpr uint32_t GROUPS = THREADS * NV;
    constexpr size_t cells = size_t(GROUPS + 2) * Traits<T>::VEC, counters = cells * (WIDE ? 4 : 2);
    a.slices = groups ? (groups + GROUPS - 1) / GROUPS : 1;
    uint64_t per_row = uint64_t(a.slices) * a.s.p;
    a.cluster = 1;
    if (share && a.r.history && a.r.history_ld >= kShareHistory && per_row > 1) {
        a.cluster = per_row < kScanCluster ? uint32_t(per_row) : kScanCluster;
        per_row = (per_row + a.cluster - 1) / a.cluster * a.cluster;
    }
    if (a.s.rows * per_row > 0x7fffffffull) return cudaErrorInvalidValue;
    a.by_row = fast_div(uint32_t(per_row));
    a.by_slices = fast_div(a.slices);
    const size_t smem = counters + (a.r.bias_count ? cells * 4 : 0);
    static std::atomic<unsigned long long> done{0};
    cudaError_t err = allow_dynamic_smem(logit_rules_kernel<T, PM, THREADS, NV, WIDE>, counters + cells * 4, L.device, done);
    if (err != cudaSuccess) return err;
    const unsigned grid = unsigned(a.s.rows * per_row);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    err = cudaLaunchKernelEx(&cfg, logit_rules_kernel<T, PM, THREADS, NV, WIDE>, a);
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
    fill_shards(&a.s, L, N.rows, N.vocab, N.ld);
    a.r = *N.rules;
    a.in_place = L.alias ? 1 : 0;
    const uint32_t groups = widest_groups<T>(a.s);
    if (N.rows * a.s.p * uint64_t(groups) < uint64_t(L.num_sms) * 1024 * PER16)
        return rules_launch<T, PM, 128, PER16, WIDE>(L, a, groups, false, info);
    return rules_launch<T, PM, 256, 4 * PER16, WIDE>(L, a, groups, true, info);
}

template <typename T>
static cudaError_t rules_dtype(const Launch &L, const RulesLaunch &N, LaunchInfo *info)
{
    // a 16-bit counter holds twice the occurrences plus one
    const bool wide = N.rules->history && N.rules->history_ld > 32767;
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
