// AllReduce fused with the residual merge and RMSNorm, with e4m3 codes and
// their scales as outputs.  Per row:
//   y = round(sum of the p rank rows), h = round(y + residual)
//   o = (h gamma) (1 / sqrt(mean(h^2) + eps)), scale = max(max |o| (1/448), 2^-126)
//   code = e4m3(o (1 / scale)), one scale for a group of columns or for the row
// As in rmsnorm.cu a cluster of C CTAs has a row, and each CTA pushes its part
// of the row's sums into every CTA of the cluster.  Multiplying by gamma before
// 1/rms makes the row's largest |o| the rounded product of its largest |h
// gamma| and 1/rms (both roundings are monotone), so that one exchange serves the mean and the row's scale;
// a group's maximum stays within lanes of a warp.
#pragma once

#include <cooperative_groups.h>
#include <math_constants.h>

#include "chunks.h"
#include "logits.cuh"

namespace ccl {

namespace cg = cooperative_groups;

constexpr int kQuantMaxCluster = 8;

template <int PM>
struct QuantArgs {
    const void *src[PM];
    void *dst[PM];
    float *scales[PM];
    uint64_t bound[PM + 1];
    uint8_t order[PM][PM];
    const void *residual;
    void *residual_out;
    const void *gamma;
    uint64_t rows;
    uint32_t hidden;
    uint32_t groups;    // scales of a row
    uint32_t lanes;     // units that share a scale; 0: the row has one
    int p;
    float eps;
    unsigned *status;
    long long wait_ns;
    int stall_test;     // 1: cluster rank 1 withholds its sums (tests); 2: the checks take every buffer for one row shorter
};

__device__ __forceinline__ uint32_t map_shared(uint32_t local, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}

__device__ __forceinline__ bool try_wait(uint32_t bar)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Waits until `bar`'s first phase is over, at most `limit` ns.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, long long limit)
{
    if (try_wait(bar)) return true;
    const uint64_t t0 = now_ns();
    while (!try_wait(bar))
        if (now_ns() - t0 > uint64_t(limit)) return false;
    return true;
}

// A load that keeps its place among the others (the buffers may be written in
// place, by the thread that read them).
__device__ __forceinline__ uint4 load_v4(const void *p)
{
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// The largest size; NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The scale of a group whose largest |o| is m.
__device__ __forceinline__ float scale_of(float m)
{
    const float s = __fmul_rn(m, 1.0f / 448.0f);
    return s < 0x1p-126f ? 0x1p-126f : s;      // (NaN stays NaN)
}

// Checked build: an access lies in the row [row, row + bytes) of a buffer, or is recorded and not made.
template <bool CHECKED>
struct RowCheck {
    __device__ static __forceinline__ RowCheck of(const void *, uint64_t, unsigned *) { return {}; }
    __device__ __forceinline__ bool holds(const void *, uint32_t) const { return true; }
};
template <>
struct RowCheck<true> {
    const void *row;
    uint64_t bytes;
    unsigned *status;
    __device__ static __forceinline__ RowCheck of(const void *row, uint64_t bytes, unsigned *status) { return {row, bytes, status}; }
    __device__ __forceinline__ bool holds(const void *at, uint32_t n) const { return in_buffer(at, n, row, bytes, status, kSiteNorm); }
};

// The VEC columns of a unit, as pairs.  VECTOR: they follow one another.  Other
// rows are read element by element, so that the 32 lanes of a load take neighbouring columns: unit u of
// a warp's 32 has every 32nd column of their 32 VEC.
template <typename T, bool VECTOR>
struct QuantUnit {
    using Tr = Traits<T>;
    using Check = RowCheck<kBoundsCheck>;
    static constexpr int VEC = Tr::VEC, S = 16 / VEC, PAIRS = VEC / 2;
    __device__ static __forceinline__ void unpack(const uint4 &v, Pair (&f)[PAIRS])
    {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) f[i] = Group<T>::pair(v, i);
    }
    __device__ static __forceinline__ uint32_t column(uint32_t u, int i) { return VECTOR ? u * VEC + i : u / 32 * (32 * VEC) + i * 32 + u % 32; }
    // unit u of the row that begins at `row`, of `hidden` columns
    __device__ static __forceinline__ uint4 load(const void *row, uint32_t u, uint32_t hidden, Check check)
    {
        if constexpr (VECTOR) {
            const char *at = static_cast<const char *>(row) + uint64_t(u) * 16;
            return check.holds(at, 16) ? load_v4(at) : make_uint4(0, 0, 0, 0);
        } else {
            float f[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = column(u, i) < hidden && check.holds(static_cast<const char *>(row) + uint64_t(column(u, i)) * S, S) ? Tr::load1(row, column(u, i)) : 0.0f;
            return Tr::pack(f);
        }
    }
    __device__ static __forceinline__ void store(void *row, uint32_t u, uint32_t hidden, const uint4 &v, Check check)
    {
        if constexpr (VECTOR) {
            char *at = static_cast<char *>(row) + uint64_t(u) * 16;
            if (check.holds(at, 16)) st_v4(at, v);
        } else {
            float f[VEC];
            Tr::unpack(v, f);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (column(u, i) < hidden && check.holds(static_cast<char *>(row) + uint64_t(column(u, i)) * S, S)) Tr::store1(row, column(u, i), f[i]);
        }
    }
    __device__ static __forceinline__ void store_codes(void *row, uint32_t u, uint32_t hidden, const uint32_t (&w)[VEC / 4], Check check)
    {
        char *to = static_cast<char *>(row) + (VECTOR ? uint64_t(u) * VEC : 0);
        if (VECTOR && !check.holds(to, VEC)) return;
        if constexpr (VECTOR && VEC == 8) {
            asm volatile("st.global.cs.v2.u32 [%0], {%1, %2};" ::"l"(to), "r"(w[0]), "r"(w[1]) : "memory");
        } else if constexpr (VECTOR) {
            asm volatile("st.global.cs.u32 [%0], %1;" ::"l"(to), "r"(w[0]) : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (column(u, i) < hidden && check.holds(to + column(u, i), 1)) to[column(u, i)] = char(w[i / 4] >> (i % 4 * 8));
        }
    }
};

// A thread has a unit of VEC columns at a time; KEEP of them stay in shared
// memory between the passes, further ones are read again.  VECTOR: units are
// 16-byte groups.  Bound by memory and by how many rows are under way: 4000 x
// 8192 f16 p=4 in 85 us (6.1 TB/s), 4096 x 8192 bf16 p=8 153 (6.2), 4096 x 4096
// bf16 p=1 21 with a scale a row, 24 with scales of 128 columns (4.8; 32768 rows 168, 5.6).  With the units in registers
// instead, at four CTAs of 256 threads an SM, of then 86, 153 and 27 us 93, 158 and 31.  Here 2048 threads an SM, or 1536 where
// four or eight ranks' loads are in registers at once (p=4 with 2048: 90, p=8 172, they spill).  A rank count of the launch
// and odd rows go rank by rank and keep 2048, although they spill 100 to 450 bytes: us with 2048 / 1536 / 1024,
//   4096 x 4096 bf16 p=5 69 / 67 / 72, p=6 74 / 76 / 83, p=7 84 / 85 / 93, p=16 145 / 152 / 156, p=64 537 / 567 / 544
//   20000 x 2001 bf16 p=1 169 / 183 / 233, 4000 x 1001 f32 p=4 41 / 49 / 60, 40000 x 301 bf16 p=1 56 / 53 / 57
// Loading two or four units at once cost more CTAs than it gained.
template <typename T, int P, int THREADS, int KEEP, bool VECTOR>
__global__ void __launch_bounds__(THREADS, KEEP > 1 ? (P >= 4 ? 1536 : 2048) / THREADS : 1) ar_rmsnorm_e4m3_kernel(const __grid_constant__ QuantArgs<(P > 0 ? P : kMaxRanks)> a)
{
    using U = QuantUnit<T, VECTOR>;
    constexpr int VEC = U::VEC, S = U::S, PAIRS = U::PAIRS, WARPS = THREADS / 32;
    __shared__ float2 red[WARPS];
    __shared__ float2 row_s;            // 1/rms, the row's largest |o|
    __shared__ __align__(8) float2 parts[kQuantMaxCluster];
    __shared__ __align__(8) uint64_t xbar;
    __shared__ bool gave_up;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), q = int(cluster.block_rank());
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t bar = uint32_t(__cvta_generic_to_shared(&xbar));
    if (C > 1) {
        // the barrier is there before a peer signals it: arrive now, wait before the first remote write
        if (threadIdx.x == 0) {
            gave_up = false;
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    grid_dependency_wait();
    grid_dependents_launch();
    const int p = P > 0 ? P : a.p;
    const uint32_t H = a.hidden, units = VECTOR ? H / VEC : (H + 32 * VEC - 1) / (32 * VEC) * 32;
    const uint64_t row = C > 1 ? blockIdx.x / C : blockIdx.x, base = row * H;
    // checked build: the row's `element` bytes a column at `at`, none where the debug hook takes the buffers to lack the row;
    // gamma's; a scale's number
    const bool held = !kBoundsCheck || row < a.rows - (a.stall_test == 2 ? 1 : 0);
    auto in_row = [&](const void *at, uint32_t element) { return U::Check::of(at, held ? uint64_t(H) * element : 0, a.status); };
    const auto in_gamma = U::Check::of(a.gamma, uint64_t(H) * S, a.status);
    auto scale_held = [&](uint32_t group) { return in_bounds(held && group < a.groups, a.status, kSiteNorm, group); };
    // this CTA's units: whole warps of them, so that the lanes that share a scale are in one warp
    const uint32_t blocks = (units + 31) / 32;
    const uint32_t u0 = C > 1 ? uint32_t(uint64_t(blocks) * q / C) * 32 : 0;
    const uint32_t u1 = C > 1 ? min(units, uint32_t(uint64_t(blocks) * (q + 1) / C) * 32) : units;
    const char *residual = static_cast<const char *>(a.residual) + base * S;
    char *merged = static_cast<char *>(a.residual_out) + base * S;

    // most rows lie in one chunk
    int chunk = 0;
    for (int hi = p; hi - chunk > 1;) {
        const int mid = (chunk + hi) / 2;
        if (base >= a.bound[mid]) chunk = mid;
        else hi = mid;
    }
    const bool one_chunk = base + H <= a.bound[chunk + 1];
    // the chunk of element e of the buffers, of this row
    auto chunk_of = [&](uint64_t e) {
        int lo = chunk;
        if (one_chunk) return lo;
        if constexpr (KEEP > 1) {      // many rows: two chunks, seldom more
            lo = chunk_from(a.bound, lo, e);
        } else {
            for (int hi = p; hi - lo > 1;) {
                const int mid = (lo + hi) / 2;
                if (e >= a.bound[mid]) lo = mid;
                else hi = mid;
            }
        }
        return lo;
    };
    // the row of the k-th rank that chunk c folds
    auto source = [&](int c, int k) -> const void * { return static_cast<const char *>(a.src[a.order[c][k]]) + base * S; };
    auto load_source = [&](int c, int k, uint32_t u) { return U::load(source(c, k), u, H, in_row(source(c, k), S)); };
    Pair ss = {0.0f, 0.0f};
    float top = 0.0f;
    // pass 1: fold, merge, store h, add its squares and find the largest |h gamma|
    auto merge = [&](uint32_t u, Pair (&acc)[PAIRS], const uint4 &res) -> uint4 {
        Pair v[PAIRS];
        if constexpr (P != 1) U::unpack(Group<T>::pack(acc), acc);       // y, rounded
        U::unpack(res, v);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) acc[i] = acc[i] + v[i];          // the merge
        const uint4 h = Group<T>::pack(acc);
        U::store(merged, u, H, h, in_row(merged, S));
        U::unpack(h, acc);                                               // h, rounded
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) ss = fma(acc[i], acc[i], ss);
        if (a.lanes == 0) {
            U::unpack(U::load(a.gamma, u, H, in_gamma), v);
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const Pair o = acc[i] * v[i];
                top = max_abs(top, o.x, o.y);
            }
        }
        return h;
    };
    // a unit element by element, each in its own chunk's order
    auto fold_elements = [&](uint32_t u, int c, Pair (&acc)[PAIRS]) {
        float f[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const uint64_t e = base + U::column(u, i);
            f[i] = 0.0f;
            if (U::column(u, i) >= H) continue;
            while (e >= a.bound[c + 1]) ++c;
            auto held_source = [&](int k) { return in_row(source(c, k), S).holds(static_cast<const char *>(a.src[a.order[c][k]]) + e * S, S); };
            if (!held_source(0)) continue;
            f[i] = Traits<T>::load1(a.src[a.order[c][0]], e);
            for (int k = 1; k < p; ++k)
                if (held_source(k)) f[i] = __fadd_rn(f[i], Traits<T>::load1(a.src[a.order[c][k]], e));
        }
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) acc[i] = {f[2 * i], f[2 * i + 1]};
    };
    auto pass1 = [&](uint32_t u, uint4 *kept) {
        if (u >= u1) return;
        Pair acc[PAIRS], v[PAIRS];
        uint4 res;
        const int c = chunk_of(base + (VECTOR ? U::column(u, 0) : lookup_column(U::column(u, 0), H)));
        if (!in_bounds(c < p, a.status, kSiteNorm, uint64_t(c))) return;
        if (!one_chunk && (!VECTOR || base + (uint64_t(u) + 1) * VEC > a.bound[c + 1])) {
            fold_elements(u, c, acc);
            res = U::load(residual, u, H, in_row(residual, S));
        } else if constexpr (P > 0) {
            uint4 r[P];
#pragma unroll
            for (int k = 0; k < P; ++k) r[k] = load_source(c, k, u);
            res = U::load(residual, u, H, in_row(residual, S));
            U::unpack(r[0], acc);
#pragma unroll
            for (int k = 1; k < P; ++k) {
                U::unpack(r[k], v);
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) acc[i] = acc[i] + v[i];
            }
        } else if constexpr (THREADS == 128 && KEEP == 1 && VECTOR) {
            // few rows: the loads of eight ranks go out before the first is folded (4 x 4096 bf16 p=64 51 -> 17 us, with its chunks found by halving); with many
            // rows their registers would cost CTAs (15683 x 2056 bf16 p=3, four at once: 144 us, one by one 108)
            res = U::load(residual, u, H, in_row(residual, S));
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) acc[i] = {0.0f, 0.0f};
            for (int k = 0; k < p; k += 8) {
                uint4 r[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) r[i] = load_source(c, min(k + i, p - 1), u);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (k + i >= p) break;
                    U::unpack(r[i], v);
#pragma unroll
                    for (int j = 0; j < PAIRS; ++j) acc[j] = k + i == 0 ? v[j] : acc[j] + v[j];
                }
            }
        } else {
            U::unpack(load_source(c, 0, u), acc);
#pragma unroll 4
            for (int k = 1; k < p; ++k) {
                U::unpack(load_source(c, k, u), v);
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) acc[i] = acc[i] + v[i];
            }
            res = U::load(residual, u, H, in_row(residual, S));
        }
        const uint4 h = merge(u, acc, res);
        if (kept) *kept = h;
    };
    const uint32_t first = u0 + threadIdx.x;
    __shared__ uint4 kept_s[KEEP][THREADS];      // each thread's own
#pragma unroll
    for (int j = 0; j < KEEP; ++j) pass1(first + j * THREADS, &kept_s[j][threadIdx.x]);
    for (uint32_t u = first + KEEP * THREADS; u < u1; u += THREADS) pass1(u, nullptr);

    // the row's sum and maximum: the warps', then (warp 0) the CTA's, then the cluster's
    float sum = ss.x + ss.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (a.lanes == 0)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, o), 0.0f);
    if (lane == 0) red[warp] = make_float2(sum, top);
    __syncthreads();
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 0) {
        const float2 mine = lane < WARPS ? red[lane] : make_float2(0.0f, 0.0f);
        sum = mine.x;
        top = mine.y;
#pragma unroll
        for (int o = WARPS / 2; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, o), 0.0f);
        }
        if (C > 1) {
            sum = __shfl_sync(0xffffffffu, sum, 0);
            top = __shfl_sync(0xffffffffu, top, 0);
            // every CTA writes its pair into parts[q] of every CTA of the row and waits for the C pairs in its own; it
            // leaves only after all writes into it have landed
            if (lane == 0)
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(uint32_t(C * 8)) : "memory");
            __syncwarp();
            if (lane < C && !(a.stall_test == 1 && q == 1))
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];"
                             ::"r"(map_shared(uint32_t(__cvta_generic_to_shared(&parts[q])), lane)), "r"(__float_as_uint(sum)),
                             "r"(__float_as_uint(top)), "r"(map_shared(bar, lane))
                             : "memory");
            if (!wait_bounded(bar, a.wait_ns)) {
                // a pair is missing: this call's outputs are wrong
                if (a.status && atomicCAS(&a.status[0], 0u, 5u) == 0u) {
                    a.status[1] = blockIdx.x;
                    a.status[2] = unsigned(row);
                    a.status[3] = threadIdx.x;
                }
                gave_up = true;
            }
            sum = 0.0f;
            top = 0.0f;
            for (int k = 0; k < C; ++k) {
                sum = __fadd_rn(sum, parts[k].x);
                top = max_abs(top, parts[k].y, 0.0f);
            }
        }
        if (lane == 0) {
            const float inv = 1.0f / sqrtf(__fadd_rn(__fdiv_rn(sum, float(H)), a.eps));
            row_s = make_float2(inv, __fmul_rn(top, inv));
        }
    }
    __syncthreads();
    const float inv = row_s.x;
    float back = 0.0f;
    if (a.lanes == 0) {
        const float scale = scale_of(row_s.y);
        back = __frcp_rn(scale);
        if (q == 0 && scale_held(0))
            // (-infinity: 1/rms is infinite, and ar_rmsnorm_e4m3_rest_kernel finds out what the scale is)
            for (int k = threadIdx.x; k < p; k += THREADS) a.scales[k][row] = inv == CUDART_INF_F && scale == inv ? -inv : scale;
    }

    // pass 2: codes to every rank.  `on`: the thread has a unit; all lanes come here together.
    auto pass2 = [&](uint32_t u, const uint4 &h, bool on) {
        Pair o[PAIRS], g[PAIRS];
        if (on) {
            U::unpack(h, o);
            U::unpack(U::load(a.gamma, u, H, in_gamma), g);
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) o[i] = o[i] * g[i] * Pair{inv, inv};
        }
        uint32_t w[VEC / 4];
        auto code = [&](const float (&by)[VEC]) {
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) {
                const Pair lo = o[2 * i] * Pair{by[4 * i], by[4 * i + 1]}, hi = o[2 * i + 1] * Pair{by[4 * i + 2], by[4 * i + 3]};
                w[i] = e4m3_pair(lo.x, lo.y) | e4m3_pair(hi.x, hi.y) << 16;
            }
        };
        float by[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) by[i] = back;
        if (a.lanes && VECTOR) {
            // the lanes of a group have its units
            float m = 0.0f;
            if (on)
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) m = max_abs(m, o[i].x, o[i].y);
            for (uint32_t l = 1; l < a.lanes; l <<= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, l), 0.0f);
            const float scale = scale_of(m), each = __frcp_rn(scale);
#pragma unroll
            for (int i = 0; i < VEC; ++i) by[i] = each;
            if (on && lane % a.lanes == 0 && scale_held(u / a.lanes)) {
                const uint64_t at = row * a.groups + u / a.lanes;
                for (int k = 0; k < p; ++k) a.scales[k][at] = scale;
            }
        } else if (a.lanes) {
            // 32 columns of a group at a time
            const uint32_t span = a.lanes * VEC / 32, block = u / 32 * VEC;
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                // (columns beyond the row are 0 times 1/rms, which may be NaN)
                if (on && U::column(u, i) < H) m = max_abs(m, i % 2 ? o[i / 2].y : o[i / 2].x, 0.0f);
                if ((i + 1) % span) continue;
#pragma unroll
                for (int l = 16; l > 0; l >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, l), 0.0f);
                const float scale = scale_of(m), each = __frcp_rn(scale);
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if (j <= i && j + int(span) > i) by[j] = each;
                const uint32_t group = (block + i) / span;
                if (group < a.groups && scale_held(group))
                    for (int k = lane; k < p; k += 32) a.scales[k][row * a.groups + group] = scale;
                m = 0.0f;
            }
        }
        if (!on) return;
        code(by);
        auto store_codes = [&](int k) {
            char *to = static_cast<char *>(a.dst[k]) + base;
            U::store_codes(to, u, H, w, in_row(to, 1));
        };
        if constexpr (P > 0) {
#pragma unroll
            for (int k = 0; k < P; ++k) store_codes(k);
        } else {
            for (int k = 0; k < p; ++k) store_codes(k);
        }
    };
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
        if (u0 + warp * 32 + j * THREADS < u1) pass2(first + j * THREADS, kept_s[j][threadIdx.x], first + j * THREADS < u1);
    for (uint32_t u = first + KEEP * THREADS; u - lane < u1; u += THREADS)
        pass2(u, u < u1 ? U::load(merged, u, H, in_row(merged, S)) : make_uint4(0, 0, 0, 0), u < u1);      // (this thread's own stores)
    if (C > 1 && gave_up) {
        // A late peer's write must not land after this CTA has gone.  The row's other CTAs come here or end, none of them
        // waits without a limit, and each has sent its pair by then; the last one's has a while to arrive.
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        wait_bounded(bar, 1000000);
    }
}

// With eps 0 a row whose mean square vanishes in fp32 has an infinite 1/rms: its products h gamma of 0 have o = NaN, which
// the largest product does not show.  A warp has a row and looks at its scale; where that is -infinity, a product of 0 makes
// it NaN, and otherwise it is infinity.  Launched for eps 0 and a scale a row alone: looking for such products in the kernel
// above cost registers that every call paid for (4096 x 16384 f32 p=3 247 -> 260 to 285 us); this costs those calls 0.8 us at
// 8 x 7168 bf16 p=8 (4.3 -> 5.1) and 12 at 100000 x 512 f32 p=1 (148 -> 160).
struct QuantRest {
    const void *merged;
    const void *gamma;
    float *scales[kMaxRanks];
    uint64_t rows, held;       // held (checked build): rows of the buffers
    uint32_t hidden;
    int p;
    unsigned *status;
};

template <typename T>
__global__ void __launch_bounds__(256) ar_rmsnorm_e4m3_rest_kernel(const __grid_constant__ QuantRest a)
{
    grid_dependency_wait();
    grid_dependents_launch();
    const uint64_t row = uint64_t(blockIdx.x) * 8 + threadIdx.x / 32;
    const uint32_t lane = threadIdx.x % 32;
    if (row >= a.rows || !in_bounds(row < a.held, a.status, kSiteNorm, row) || a.scales[0][row] != -CUDART_INF_F) return;
    bool zero = false;
    for (uint32_t c = lane; c < a.hidden; c += 32)
        zero = zero || __fmul_rn(Traits<T>::load1(a.merged, row * a.hidden + c), Traits<T>::load1(a.gamma, c)) == 0.0f;
    const float scale = __any_sync(0xffffffffu, zero) ? CUDART_NAN_F : CUDART_INF_F;
    for (int k = lane; k < a.p; k += 32) a.scales[k][row] = scale;
}

template <typename T>
static cudaError_t quant_rest(const Launch &L, const NormE4m3Launch &N, LaunchInfo *info)
{
    QuantRest a;
    a.merged = N.norm.residual_out;
    a.gamma = N.norm.gamma;
    for (int k = 0; k < L.p; ++k) a.scales[k] = N.scales[k];
    a.rows = N.norm.rows;
    a.held = N.norm.rows - (L.stall_test == 2 ? 1 : 0);
    a.hidden = uint32_t(N.norm.hidden);
    a.p = L.p;
    a.status = L.status;
    const cudaError_t err = launch_dependent(ar_rmsnorm_e4m3_rest_kernel<T>, unsigned((a.rows + 7) / 8), 256, 0, L.stream, a);
    if (err == cudaSuccess) ++info->kernels;
    return err;
}

template <typename T, int P, bool VECTOR>
static cudaError_t quant_launch(const Launch &L, const NormE4m3Launch &N, LaunchInfo *info)
{
    constexpr int PM = P > 0 ? P : kMaxRanks, VEC = Traits<T>::VEC;
    QuantArgs<PM> a;
    for (int k = 0; k < L.p; ++k) {
        a.src[k] = L.src[k];
        a.dst[k] = L.dst[k];
        a.scales[k] = N.scales[k];
    }
    for (int c = 0; c <= L.p; ++c) a.bound[c] = L.table->bound[c];
    for (int c = 0; c < L.p; ++c)
        for (int k = 0; k < L.p; ++k) a.order[c][k] = L.table->order[c * L.p + k];
    a.residual = N.norm.residual;
    a.residual_out = N.norm.residual_out;
    a.gamma = N.norm.gamma;
    a.rows = N.norm.rows;
    a.hidden = uint32_t(N.norm.hidden);
    a.groups = N.group ? uint32_t((N.norm.hidden + N.group - 1) / N.group) : 1;
    a.lanes = N.group / VEC;
    a.p = L.p;
    a.eps = N.norm.eps;
    a.status = L.status;
    a.wait_ns = L.wait_limit_ns > 0 ? L.wait_limit_ns : 2000000000LL;
    a.stall_test = L.stall_test;
    // CTA shape by rows against the SMs, as in rmsnorm.cu, and by width.  Whole groups, us (bf16 p=8, scales of 128 columns)
    // with threads x units kept of 128x1 / 1024x1 / 64x4 / 128x4 / 256x4 / 512x4:
    //   100 rows of 1536     4.5 /  4.6 /  6.6 /  5.4 /  4.2 /  4.2     4096 rows of 768    17 /  77 /  17 /  15 /  20 /  34
    //   100 rows of 8192     5.9 /  7.1 /  8.9 /  9.6 /  9.2 /  7.1     4096 rows of 1536   44 /  86 /  33 /  32 /  32 /  43
    //   200 rows of 1536     4.9 /  6.7 /  6.7 /  5.6 /  4.7 /  4.6     4096 rows of 4096  100 / 115 / 106 /  80 /  78 /  78
    //   200 rows of 8192    10.3 / 11.3 / 11.2 / 10.8 / 10.9 /  9.7     4096 rows of 8192  206 / 170 / 212 / 159 / 153 / 155
    //   300 rows of 16384     30 /   36 /   43 /   34 /   27 /   27     4096 rows of 16384 366 / 429 / 454 / 320 / 308 / 303
    // (between SMs and twice as many rows the 1024 threads of rmsnorm.cu are not the best here.)  Rows that are no 16-byte
    // groups, us with 64 / 512
    // threads (128): 2320 x 372 f16 p=1 8.9 / 21, 9217 x 499 f32 p=1 15 / 45; 914 x 1795 bf16 p=8 (128: 34) / 26.
    const uint64_t units = VECTOR ? N.norm.hidden / VEC : (N.norm.hidden + 32 * VEC - 1) / (32 * VEC) * 32, sms = uint64_t(L.num_sms), rows = N.norm.rows;
    const int threads = rows < sms      ? 128
                        : !VECTOR       ? (units <= 128 ? 64 : 512)
                        : rows < 2 * sms ? 1024
                        : units <= 256  ? 64
                        : units <= 512  ? 128
                        : units <= 1024 ? 256
                                        : 512;
    const int keep = rows < sms ? 1 : !VECTOR ? 2 : rows < 2 * sms ? 1 : 4;
    const uint64_t per_cta = uint64_t(threads) * keep;
    const uint64_t want = (units + per_cta - 1) / per_cta;
    const int C = int(want > uint64_t(kQuantMaxCluster) ? kQuantMaxCluster : want);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(rows * C));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(C);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    void (*kern)(QuantArgs<PM>) = nullptr;
    if constexpr (VECTOR) {
        kern = keep == 1 ? (threads == 128 ? ar_rmsnorm_e4m3_kernel<T, P, 128, 1, true> : ar_rmsnorm_e4m3_kernel<T, P, 1024, 1, true>)
               : threads == 64  ? ar_rmsnorm_e4m3_kernel<T, P, 64, 4, true>
               : threads == 128 ? ar_rmsnorm_e4m3_kernel<T, P, 128, 4, true>
               : threads == 512 ? ar_rmsnorm_e4m3_kernel<T, P, 512, 4, true>
                                : ar_rmsnorm_e4m3_kernel<T, P, 256, 4, true>;
    } else {
        kern = keep == 1        ? ar_rmsnorm_e4m3_kernel<T, P, 128, 1, false>
               : threads == 64  ? ar_rmsnorm_e4m3_kernel<T, P, 64, 2, false>
                                : ar_rmsnorm_e4m3_kernel<T, P, 512, 2, false>;
    }
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, a);
    if (err != cudaSuccess) return err;
    info->kernel = "allreduce_residual_rmsnorm_e4m3";
    info->grid = int(rows * C);
    info->block = threads;
    info->smem = 0;
    info->kernels = 1;
    return N.norm.eps == 0.0f && N.group == 0 ? quant_rest<T>(L, N, info) : cudaSuccess;
}

template <typename T>
static cudaError_t quant_dtype(const Launch &L, const NormE4m3Launch &N, LaunchInfo *info)
{
    if (!L.vec) return quant_launch<T, 0, false>(L, N, info);
    switch (L.p) {
    case 1: return quant_launch<T, 1, true>(L, N, info);
    case 2: return quant_launch<T, 2, true>(L, N, info);
    case 3: return quant_launch<T, 3, true>(L, N, info);
    case 4: return quant_launch<T, 4, true>(L, N, info);
    case 8: return quant_launch<T, 8, true>(L, N, info);
    default: return quant_launch<T, 0, true>(L, N, info);
    }
}

}  // namespace ccl
