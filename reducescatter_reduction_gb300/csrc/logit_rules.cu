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
// One CTA per (row, slice of the vocabulary).  It keeps one counter per token
// of its slice in shared memory, scans the row's history once and counts the
// tokens that fall into the slice (integer atomics, so any order gives the same counts),
// adds up the row's bias entries in list order, and then streams its slice:
// a 16-byte group whose counters and biases are all zero is copied through
// its mask.  Bytes: the logits once in and once out, plus the history once
// per slice (L2).
#include "logits.cuh"

namespace ccl {

template <int PM>
struct RulesArgs {
    Shards<PM> s;
    ccl_logit_rules_t r;
    uint32_t slices;     // per row
    uint32_t total;      // group slots per row
    int in_place;
};

// Generated occurrences sit above bit 0, bit 0 says "in the prompt".
constexpr uint32_t kSeenPrompt = 1, kGenerated = 2;

template <typename T, int PM, int THREADS, int NV>
__global__ void __launch_bounds__(THREADS) logit_rules_kernel(const __grid_constant__ RulesArgs<PM> a)
{
    using Tr = Traits<T>;
    constexpr int VEC = Tr::VEC;
    constexpr int SLOTS = THREADS * NV * VEC;
    extern __shared__ uint4 smem4[];
    uint32_t *cnt = reinterpret_cast<uint32_t *>(smem4);
    float *bias = reinterpret_cast<float *>(cnt + SLOTS);
    const Shards<PM> &s = a.s;
    const uint64_t row = blockIdx.x / a.slices;
    const uint32_t slice = blockIdx.x % a.slices;
    const uint32_t g0 = slice * (THREADS * NV), g1 = min(g0 + THREADS * NV, a.total);
    const bool history = a.r.history != nullptr, biased = a.r.bias_count != 0;
    const bool row_ok = row < s.rows;

    if (history)
        for (int i = threadIdx.x; i < SLOTS / 4; i += THREADS) reinterpret_cast<uint4 *>(cnt)[i] = make_uint4(0, 0, 0, 0);
    if (biased)
        for (int i = threadIdx.x; i < SLOTS / 4; i += THREADS) reinterpret_cast<uint4 *>(bias)[i] = make_uint4(0, 0, 0, 0);
    grid_dependency_wait();
    grid_dependents_launch();

    // the slice's tokens are [t0, t1): slots run through the ranks in order
    auto token_at = [&](uint32_t slot) -> uint32_t {   // first token at or after the slot's begin
        if (slot >= a.total) return s.vocab;
        const uint32_t r = rank_of_slot(s, slot), w = shard_width(s, r);
        const int e = group_begin<T>(shard_row<T>(s.in[r], s.ld, row, w), slot - r * s.nv);
        return shard_begin(s, r) + (e < 0 ? 0u : min(uint32_t(e), w));
    };
    const uint32_t t0 = token_at(g0), t1 = token_at(g1);
    auto slot_of = [&](uint32_t v) -> uint32_t {       // counter of a token of the slice
        const uint32_t r = rank_of_token(s, v);
        const ShardRow sr = shard_row<T>(s.in[r], s.ld, row, shard_width(s, r));
        return (r * s.nv - g0) * VEC + (v - shard_begin(s, r)) + sr.shift;
    };

    const uint32_t *mask = nullptr;
    uint32_t words = (s.vocab + 31) / 32;
    if (a.r.mask) {
        const int64_t m = a.r.mask_index ? int64_t(a.r.mask_index[row]) : int64_t(row);
        if (m >= 0 && m < int64_t(a.r.mask_rows)) mask = a.r.mask + uint64_t(m) * a.r.mask_ld;
    }
    __syncthreads();
    if (history) {
        const int32_t *h = a.r.history + row * a.r.history_ld;
        const int64_t ld = int64_t(a.r.history_ld);
        int64_t len = a.r.history_len ? int64_t(a.r.history_len[row]) : ld;
        len = len < 0 ? 0 : len > ld ? ld : len;
        const int64_t prompt = a.r.prompt_len ? int64_t(a.r.prompt_len[row]) : 0;
        for (int64_t j = threadIdx.x; j < len; j += THREADS) {
            const uint32_t v = uint32_t(h[j]);
            if (v - t0 >= t1 - t0) continue;           // also a negative token, or one past the vocabulary
            uint32_t *c = &cnt[slot_of(v)];
            if (j < prompt) atomicOr(c, kSeenPrompt);
            else atomicAdd(c, kGenerated);
        }
    }
    if (biased && threadIdx.x < 32) {
        // one warp, 32 entries at a time: entries of one token add in list order
        const int64_t n = int64_t(a.r.bias_count);
        int64_t lo = a.r.bias_offsets[row], hi = a.r.bias_offsets[row + 1];
        lo = lo < 0 ? 0 : lo > n ? n : lo;
        hi = hi < lo ? lo : hi > n ? n : hi;
        for (int64_t b = lo; b < hi; b += 32) {
            const int64_t k = b + threadIdx.x;
            const uint32_t v = k < hi ? uint32_t(a.r.bias_tokens[k]) : 0xffffffffu;
            const bool mine = k < hi && v - t0 < t1 - t0;
            const float add = mine ? a.r.bias_values[k] : 0.0f;
            const unsigned same = __match_any_sync(0xffffffffu, mine ? v : 0xffffffffu);
            const int turn = mine ? __popc(same & ((1u << threadIdx.x) - 1)) : -1;
            float *at = mine ? &bias[slot_of(v)] : bias;
            for (int t = 0; __any_sync(0xffffffffu, turn >= t); ++t) {
                if (turn == t) *at = __fadd_rn(*at, add);
                __syncwarp();
            }
        }
    }
    __syncthreads();

    const float rep = a.r.repetition ? a.r.repetition[row] : 1.0f;
    const float freq = a.r.frequency ? a.r.frequency[row] : 0.0f;
    const float pres = a.r.presence ? a.r.presence[row] : 0.0f;
    constexpr uint32_t ALL = (1u << VEC) - 1;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const uint32_t local = threadIdx.x + n * THREADS, slot = g0 + local;
        if (slot >= g1) break;
        const uint32_t r = rank_of_slot(s, slot), w = shard_width(s, r), j = slot - r * s.nv;
        const ShardRow in = shard_row<T>(s.in[r], s.ld, row, w), out = shard_row<T>(s.out[r], s.ld, row, w);
        const int e = group_begin<T>(in, j);
        if (e >= int(w)) continue;
        uint32_t allowed = ALL;
        if (mask) {
            // bits [v, v + VEC) of the row's mask, two words at most; a bit before the shard's first token is unused
            const int v = int(shard_begin(s, r)) + e;
            const uint32_t at = v < 0 ? 0u : uint32_t(v);
            const uint32_t lo = mask[at >> 5], hi = (at >> 5) + 1 < words ? mask[(at >> 5) + 1] : 0u;
            allowed = __funnelshift_r(lo, hi, at & 31);
            if (v < 0) allowed <<= -v;
            allowed &= ALL;
        }
        uint32_t c[VEC], any = 0;
        float b[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            c[i] = history ? cnt[local * VEC + i] : 0u;
            b[i] = biased ? bias[local * VEC + i] : 0.0f;
            any |= c[i] | (b[i] != 0.0f ? 1u : 0u);
        }
        if (a.in_place && !any && allowed == ALL) continue;
        float x[VEC];
        Tr::unpack(load_group<T>(in, j, row_ok, s.status, kSiteRules), x);
        if (any) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if (b[i] != 0.0f) x[i] = __fadd_rn(x[i], b[i]);
                if (c[i]) x[i] = x[i] > 0.0f ? __fdiv_rn(x[i], rep) : __fmul_rn(x[i], rep);
                if (c[i] >= kGenerated) x[i] = __fsub_rn(__fsub_rn(x[i], __fmul_rn(freq, float(c[i] >> 1))), pres);
            }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (!((allowed >> i) & 1)) x[i] = -INFINITY;
        store_group<T>(out, in, j, Tr::pack(x), row_ok, s.status, kSiteRules);
    }
}

template <typename T, int PM, int THREADS, int NV>
static cudaError_t rules_launch(const Launch &L, RulesArgs<PM> &a, LaunchInfo *info)
{
    constexpr uint32_t GROUPS = THREADS * NV;
    constexpr size_t table = size_t(GROUPS) * Traits<T>::VEC * 4;
    a.slices = (a.total + GROUPS - 1) / GROUPS;
    const size_t smem = (a.r.bias_count ? 2 : 1) * table;
    if (a.s.rows * a.slices > 0x7fffffffull) return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> done{0};
    cudaError_t err = allow_dynamic_smem(logit_rules_kernel<T, PM, THREADS, NV>, 2 * table, L.device, done);
    if (err != cudaSuccess) return err;
    const unsigned grid = unsigned(a.s.rows * a.slices);
    err = launch_dependent(logit_rules_kernel<T, PM, THREADS, NV>, grid, THREADS, smem, L.stream, a);
    if (err != cudaSuccess) return err;
    info->kernel = "logit_rules";
    info->grid = int(grid);
    info->block = THREADS;
    info->smem = smem;
    info->kernels = 1;
    return cudaGetLastError();
}

template <typename T, int PM>
static cudaError_t rules_shape(const Launch &L, const RulesLaunch &N, LaunchInfo *info)
{
    constexpr int PER16 = Traits<T>::VEC == 8 ? 1 : 2;   // groups that hold eight elements
    RulesArgs<PM> a;
    fill_shards(&a.s, L, N.rows, N.vocab, N.ld);
    a.r = *N.rules;
    a.in_place = L.alias ? 1 : 0;
    a.total = a.s.p * a.s.nv;
    const uint64_t groups = N.rows * uint64_t(a.total);
    if (groups < uint64_t(L.num_sms) * 1024 * PER16) return rules_launch<T, PM, 128, PER16>(L, a, info);
    return rules_launch<T, PM, 512, 2 * PER16>(L, a, info);
}

template <typename T>
static cudaError_t rules_dtype(const Launch &L, const RulesLaunch &N, LaunchInfo *info)
{
    return L.p == 1 ? rules_shape<T, 1>(L, N, info) : L.p <= 8 ? rules_shape<T, 8>(L, N, info)
                                                               : rules_shape<T, kMaxRanks>(L, N, info);
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
