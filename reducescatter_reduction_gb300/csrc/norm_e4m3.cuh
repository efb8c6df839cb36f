// AllReduce fused with the residual merge and RMSNorm, with e4m3 codes and
// their scales as outputs.  Per row:
//   y = round(sum of the p rank rows), h = round(y + residual)
//   o = (h gamma) (1 / sqrt(mean(h^2) + eps)), scale = max(max |o| / 448, 2^-126)
//   code = e4m3(o / scale), one scale for a group of columns or for the row
// As in rmsnorm.cu a cluster of C CTAs has a row, and each CTA pushes its part
// of the row's sums into every CTA of the cluster.  Multiplying by gamma before
// 1/rms makes the row's largest |o| the rounded product of its largest |h
// gamma| and 1/rms (both roundings are monotone), so that one exchange serves the mean and the row's scale;
// a group's maximum stays within lanes of a warp.
#pragma once

#include <cooperative_groups.h>

#include "device.cuh"

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
    uint64_t rows, hidden;
    uint32_t groups;    // scales of a row
    uint32_t lanes;     // lanes of a warp that share a scale; 0: the row has one
    int p;
    int vec;            // 16-byte groups: pointers aligned, hidden and every chunk boundary multiples of VEC
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

// The larger; NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
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
    const float s = __fdiv_rn(m, 448.0f);
    return s < 0x1p-126f ? 0x1p-126f : s;      // (NaN stays NaN)
}

// One unit, VEC columns of a row, a thread at a time.
template <typename T, int P, int THREADS, int KEEP>
__global__ void __launch_bounds__(THREADS) ar_rmsnorm_e4m3_kernel(const __grid_constant__ QuantArgs<(P > 0 ? P : kMaxRanks)> a)
{
    using Tr = Traits<T>;
    using F = Fold<T, OP_SUM>;
    constexpr int VEC = Tr::VEC, S = 16 / VEC, WARPS = THREADS / 32;
    __shared__ float2 red[32];
    __shared__ __align__(8) float2 parts[kQuantMaxCluster];
    __shared__ __align__(8) uint64_t xbar;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), q = int(cluster.block_rank());
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t bar = uint32_t(__cvta_generic_to_shared(&xbar));
    if (C > 1) {
        // the barrier is there before a peer signals it: arrive now, wait before the first remote write
        if (threadIdx.x == 0) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    grid_dependency_wait();
    grid_dependents_launch();
    const int p = P > 0 ? P : a.p;
    const uint64_t H = a.hidden, row = blockIdx.x / C, base = row * H;
    const uint64_t held = (a.rows - (a.stall_test == 2 ? 1 : 0)) * H;       // (checked build)
    // this CTA's columns: whole warps of units, so that the lanes that share a scale are in one warp
    const uint64_t blocks = (H + 32 * VEC - 1) / (32 * VEC);
    const uint64_t b0 = blocks * q / C, b1 = blocks * (q + 1) / C;

    auto load_unit = [&](const void *buf, uint64_t c, uint64_t at, float (&f)[VEC]) {    // columns c ... from element `at`
        if (a.vec) {
            Tr::unpack(ld_coherent_v4(static_cast<const char *>(buf) + at * S), f);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = c + i < H ? Tr::load1(buf, at + i) : 0.0f;
        }
    };
    float ss = 0.0f, top = 0.0f;
    // pass 1: fold, merge, store h, its squares and largest |h gamma|
    auto pass1 = [&](uint64_t b) -> uint4 {
        const uint64_t c = (b * 32 + lane) * VEC, e = base + c;
        const uint64_t end = c + VEC < H ? c + VEC : H;
        if (c >= H || !in_bounds(base + end <= held, a.status, kSiteNorm, e)) return make_uint4(0, 0, 0, 0);
        float acc[VEC], v[VEC];
        if (a.vec) {
            int ch = 0;
            while (e >= a.bound[ch + 1]) ++ch;
            if constexpr (P > 0) {
                uint4 r[P];
#pragma unroll
                for (int k = 0; k < P; ++k) r[k] = ld_coherent_v4(static_cast<const char *>(a.src[a.order[ch][k]]) + e * S);
                if constexpr (THREADS <= 128) hold_batch(r);
                Tr::unpack(r[0], acc);
#pragma unroll
                for (int k = 1; k < P; ++k) {
                    Tr::unpack(r[k], v);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) acc[i] = F::fold(acc[i], v[i], 1.0f);
                }
            } else {
                Tr::unpack(ld_coherent_v4(static_cast<const char *>(a.src[a.order[ch][0]]) + e * S), acc);
                for (int k = 1; k < p; ++k) {
                    Tr::unpack(ld_coherent_v4(static_cast<const char *>(a.src[a.order[ch][k]]) + e * S), v);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) acc[i] = F::fold(acc[i], v[i], 1.0f);
                }
            }
        } else {
            int ch = 0;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                acc[i] = 0.0f;
                if (c + i >= H) continue;
                while (e + i >= a.bound[ch + 1]) ++ch;
                acc[i] = Tr::load1(a.src[a.order[ch][0]], e + i);
                for (int k = 1; k < p; ++k) acc[i] = F::fold(acc[i], Tr::load1(a.src[a.order[ch][k]], e + i), 1.0f);
            }
        }
        Tr::unpack(Tr::pack(acc), acc);                                  // y, rounded
        load_unit(a.residual, c, e, v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = __fadd_rn(acc[i], v[i]);   // the merge
        const uint4 h = Tr::pack(acc);
        Tr::unpack(h, acc);                                              // h, rounded
        if (a.vec) {
            st_v4(static_cast<char *>(a.residual_out) + e * S, h);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (c + i < H) Tr::store1(a.residual_out, e + i, acc[i]);
        }
        load_unit(a.gamma, c, c, v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            ss = __fadd_rn(ss, __fmul_rn(acc[i], acc[i]));
            top = max_nan(top, fabsf(__fmul_rn(acc[i], v[i])));
        }
        return h;
    };
    uint4 keep[KEEP];
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
        const uint64_t b = b0 + warp + uint64_t(j) * WARPS;
        if (b < b1) keep[j] = pass1(b);
    }
    for (uint64_t b = b0 + warp + uint64_t(KEEP) * WARPS; b < b1; b += WARPS) pass1(b);

    // the row's sum and maximum
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (lane == 0) red[warp] = make_float2(ss, top);
    __syncthreads();
    ss = 0.0f;
    top = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        ss = __fadd_rn(ss, red[w].x);
        top = max_nan(top, red[w].y);
    }
    if (C > 1) {
        // every CTA writes its pair into parts[q] of every CTA of the row and waits for the C pairs in its own; it
        // leaves only after all writes into it have landed
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (threadIdx.x == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(uint32_t(C * 8)) : "memory");
        if (int(threadIdx.x) < C && !(a.stall_test == 1 && q == 1))
            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];"
                         ::"r"(map_shared(uint32_t(__cvta_generic_to_shared(&parts[q])), threadIdx.x)), "r"(__float_as_uint(ss)),
                         "r"(__float_as_uint(top)), "r"(map_shared(bar, threadIdx.x))
                         : "memory");
        if (!wait_bounded(bar, a.wait_ns)) {
            // A pair is missing (this call's outputs are wrong).  Once more, again bounded, so that a late peer's write
            // does not land after this CTA has gone.
            if (a.status && atomicCAS(&a.status[0], 0u, 5u) == 0u) {
                a.status[1] = blockIdx.x;
                a.status[2] = unsigned(row);
                a.status[3] = threadIdx.x;
            }
            wait_bounded(bar, a.wait_ns);
        }
        ss = 0.0f;
        top = 0.0f;
        for (int k = 0; k < C; ++k) {
            ss = __fadd_rn(ss, parts[k].x);
            top = max_nan(top, parts[k].y);
        }
    }
    const float inv = 1.0f / sqrtf(__fadd_rn(__fdiv_rn(ss, float(H)), a.eps));
    const float row_scale = scale_of(__fmul_rn(top, inv));
    if (a.lanes == 0 && q == 0)
        for (int k = threadIdx.x; k < p; k += THREADS)
            if (in_bounds(base + H <= held, a.status, kSiteNorm, row)) a.scales[k][row] = row_scale;

    // pass 2: codes to every rank
    auto pass2 = [&](uint64_t b, const uint4 &h) {
        const uint64_t c = (b * 32 + lane) * VEC, e = base + c;
        const uint64_t end = c + VEC < H ? c + VEC : H;
        const bool has = c < H && in_bounds(base + end <= held, a.status, kSiteNorm, e);
        float o[VEC], g[VEC];
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = 0.0f;
        if (has) {
            Tr::unpack(h, o);
            load_unit(a.gamma, c, c, g);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                o[i] = __fmul_rn(__fmul_rn(o[i], g[i]), inv);
                if (a.vec || c + i < H) m = max_nan(m, fabsf(o[i]));
            }
        }
        float scale = row_scale;
        if (a.lanes) {
            for (uint32_t l = 1; l < a.lanes; l <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, l));
            scale = scale_of(m);
            if (has && lane % a.lanes == 0) {
                const uint64_t at = row * a.groups + c / (a.lanes * VEC);
                for (int k = 0; k < p; ++k) a.scales[k][at] = scale;
            }
        }
        if (!has) return;
        uint32_t w[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            w[i] = e4m3_pair(__fdiv_rn(o[4 * i], scale), __fdiv_rn(o[4 * i + 1], scale)) |
                   e4m3_pair(__fdiv_rn(o[4 * i + 2], scale), __fdiv_rn(o[4 * i + 3], scale)) << 16;
        auto store = [&](void *dst) {
            char *to = static_cast<char *>(dst) + e;
            if (a.vec) {
                if constexpr (VEC == 8) asm volatile("st.global.cs.v2.u32 [%0], {%1, %2};" ::"l"(to), "r"(w[0]), "r"(w[1]) : "memory");
                else asm volatile("st.global.cs.u32 [%0], %1;" ::"l"(to), "r"(w[0]) : "memory");
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (c + i < H) to[i] = char(w[i / 4] >> (i % 4 * 8));
            }
        };
        if constexpr (P > 0) {
#pragma unroll
            for (int k = 0; k < P; ++k) store(a.dst[k]);
        } else {
            for (int k = 0; k < p; ++k) store(a.dst[k]);
        }
    };
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
        const uint64_t b = b0 + warp + uint64_t(j) * WARPS;
        if (b < b1) pass2(b, keep[j]);
    }
    for (uint64_t b = b0 + warp + uint64_t(KEEP) * WARPS; b < b1; b += WARPS) {
        const uint64_t c = (b * 32 + lane) * VEC;
        uint4 h = make_uint4(0, 0, 0, 0);
        const uint64_t end = c + VEC < H ? c + VEC : H;
        if (c < H && in_bounds(base + end <= held, a.status, kSiteNorm, base + c)) {
            float f[VEC];
            load_unit(a.residual_out, c, base + c, f);      // (this thread's own stores)
            h = Tr::pack(f);
        }
        pass2(b, h);
    }
}

template <typename T, int P>
static cudaError_t quant_launch(const Launch &L, const NormE4m3Launch &N, LaunchInfo *info)
{
    constexpr int PM = P > 0 ? P : kMaxRanks, VEC = Traits<T>::VEC;
    QuantArgs<PM> a = {};
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
    a.hidden = N.norm.hidden;
    a.groups = N.group ? uint32_t((N.norm.hidden + N.group - 1) / N.group) : 1;
    a.lanes = N.group / VEC;
    a.p = L.p;
    a.vec = L.vec ? 1 : 0;
    a.eps = N.norm.eps;
    a.status = L.status;
    a.wait_ns = L.wait_limit_ns > 0 ? L.wait_limit_ns : 2000000000LL;
    a.stall_test = L.stall_test;
    // the shapes of rmsnorm.cu: decode, one to two rows an SM, prefill
    const uint64_t blocks = (N.norm.hidden + 32 * VEC - 1) / (32 * VEC), sms = uint64_t(L.num_sms), rows = N.norm.rows;
    const int threads = rows < sms ? 128 : rows < 2 * sms ? 1024 : 256;
    const uint64_t per_cta = uint64_t(threads / 32) * (rows < 2 * sms ? 1 : 4);
    const uint64_t want = (blocks + per_cta - 1) / per_cta;
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
    const cudaError_t err = threads == 128    ? cudaLaunchKernelEx(&cfg, ar_rmsnorm_e4m3_kernel<T, P, 128, 1>, a)
                            : threads == 1024 ? cudaLaunchKernelEx(&cfg, ar_rmsnorm_e4m3_kernel<T, P, 1024, 1>, a)
                                              : cudaLaunchKernelEx(&cfg, ar_rmsnorm_e4m3_kernel<T, P, 256, 4>, a);
    if (err != cudaSuccess) return err;
    info->kernel = "allreduce_residual_rmsnorm_e4m3";
    info->grid = int(rows * C);
    info->block = threads;
    info->smem = 0;
    info->kernels = 1;
    return cudaSuccess;
}

template <typename T>
static cudaError_t quant_dtype(const Launch &L, const NormE4m3Launch &N, LaunchInfo *info)
{
    switch (L.p) {
    case 1: return quant_launch<T, 1>(L, N, info);
    case 2: return quant_launch<T, 2>(L, N, info);
    case 4: return quant_launch<T, 4>(L, N, info);
    case 8: return quant_launch<T, 8>(L, N, info);
    default: return quant_launch<T, 0>(L, N, info);
    }
}

}  // namespace ccl
