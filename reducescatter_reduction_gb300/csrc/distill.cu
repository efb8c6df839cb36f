// Distillation from a teacher's top K logits, the student's vocabulary split
// over the ranks: the loss, its gradient, or both in one pass.
//
// Per row, with q = softmax(t / T) over the row's valid teacher entries and
// p = softmax(z / T) over the student's vocabulary:
//   loss = T^2 sum_k q_k (log q_k - log p_{id_k})
//   dz_v = w T (p_v - sum over the k with id_k = v of q_k)
// A cluster of C CTAs takes a row, each CTA an equal part of its 16-byte
// groups.  Every thread reads its groups once, keeps exp((z - m) / T) of the
// first NV of them in registers against its own maximum m, and after the
// exchange of (max, sum, the teacher's share of the loss) between the CTAs
// scales them into the gradient: the logits are read once and the gradient
// written once, 2 R V s bytes, with one exponential per element.  Groups past
// the first NV per thread (vocabularies beyond C * THREADS * NV groups) are
// read a second time.  The teacher's entries are then put right one by one:
// after the CTA's barrier, the thread of an entry's first occurrence stores
// the gradient of that token with the teacher's share taken off.
//
// The CTAs of a row exchange their sums by writing them into one another's
// shared memory before the cluster's hardware barrier; every CTA adds the
// same C values in the same order, so all parts of a row use the same bits.
// Differences z - m are formed before the scaling by 1 / T, so that masks of
// the type's lowest value do not turn into inf - inf.
#include "logits.cuh"

namespace ccl {

constexpr int kDistillMaxCluster = 8;

template <int PM>
struct DistillArgs {
    Shards<PM> s;
    const int32_t *ids;
    const void *teacher;
    const float *weight;
    float *loss;
    float *stats;
    float temperature;
    float to_log2;       // log2(e) / T
    uint32_t k, kpad;
    uint32_t cluster;    // CTAs per row
    uint32_t total;      // group slots per row
    int teacher_dtype;
};

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A maximum of nothing but -inf: differences to it are formed against 0, so
// that exp gives 0 and not NaN.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.0f : m; }

__device__ __forceinline__ float load_any(const void *p, int dtype, uint64_t i)
{
    return dtype == DT_F32 ? Traits<F32>::load1(p, i) : dtype == DT_F16 ? Traits<F16>::load1(p, i) : Traits<BF16>::load1(p, i);
}

// What one CTA of a row tells the others.
struct Part {
    float m, s;      // its maximum, sum exp((z - m) / T)
    float dot, own;  // over the teacher's entries in its columns: sum e_k (z - m), sum e_k
};

template <typename T, int PM, int PASS, int THREADS, int NV>
__global__ void __launch_bounds__(THREADS) distill_kernel(const __grid_constant__ DistillArgs<PM> a)
{
    using Tr = Traits<T>;
    constexpr int VEC = Tr::VEC;
    constexpr int WARPS = THREADS / 32;
    constexpr bool FWD = PASS & CCL_PASS_FORWARD, BWD = PASS & CCL_PASS_BACKWARD;
    extern __shared__ uint4 smem4[];
    int *id_s = reinterpret_cast<int *>(smem4);                    // ids, -1 where there is none
    float *e_s = reinterpret_cast<float *>(id_s + a.kpad);         // exp((t - tmax) / T)
    float *z_s = e_s + a.kpad;                                     // the student's logits at the ids in these columns
    __shared__ float red[8][WARPS];
    __shared__ float4 parts[kDistillMaxCluster];
    const Shards<PM> &s = a.s;
    const uint32_t C = a.cluster, q = blockIdx.x % C;
    const uint64_t row = blockIdx.x / C;
    const bool row_ok = row < s.rows;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (FWD && C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    grid_dependency_wait();
    grid_dependents_launch();

    const uint32_t g0 = uint32_t(uint64_t(a.total) * q / C), g1 = uint32_t(uint64_t(a.total) * (q + 1) / C);
    auto in_row = [&](uint32_t r) { return shard_row<T>(s.in[r], s.ld, row, shard_width(s, r)); };
    auto load = [&](uint32_t slot) -> uint4 {
        const uint32_t r = rank_of_slot(s, slot);
        return load_group<T>(in_row(r), slot - r * s.nv, row_ok, s.status, kSiteDistill);
    };
    const uint32_t low = VEC == 4 ? 0xff800000u : Tr::kDtype == DT_BF16 ? 0xff80ff80u : 0xfc00fc00u;   // -inf
    uint4 raw[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const uint32_t slot = g0 + tid + n * THREADS;
        raw[n] = slot < g1 ? load(slot) : make_uint4(low, low, low, low);
    }

    // the teacher's entries
    float tm = -INFINITY;
    for (uint32_t k = tid; k < a.kpad; k += THREADS) {
        int id = k < a.k ? a.ids[row * a.k + k] : -1;
        if (uint32_t(id) >= s.vocab) id = -1;
        float t = -INFINITY, z = 0.0f;
        if (id >= 0) {
            t = load_any(a.teacher, a.teacher_dtype, row * a.k + k);
            const uint32_t r = rank_of_token(s, uint32_t(id));
            const ShardRow sr = in_row(r);
            const uint32_t at = uint32_t(id) - shard_begin(s, r) + sr.shift;
            const uint32_t slot = r * s.nv + at / VEC;
            // an entry of another CTA's columns keeps its id, with the sign bit set
            if (slot >= g0 && slot < g1) {
                if (in_bounds(row_ok, s.status, kSiteDistill, id)) z = Tr::load1(reinterpret_cast<const void *>(sr.base), at);
            } else {
                id |= int(0x80000000u);
            }
        }
        id_s[k] = id;
        e_s[k] = t;
        z_s[k] = z;
        tm = fmaxf(tm, t);
    }

    // this thread's maximum and sum; e holds the first NV groups' exponentials
    hold_batch(raw);
    float e[NV * VEC];
    float m = -INFINITY, sum = 0.0f;
    const float c2 = a.to_log2;
    float row_m = 0.0f, inv = 0.0f;
    if constexpr (FWD) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float f[VEC];
            Tr::unpack(raw[n], f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                e[n * VEC + i] = f[i];
                m = fmaxf(m, f[i]);
            }
        }
    } else {
        row_m = finite_max(a.stats[2 * row]);
        inv = a.stats[2 * row] == -INFINITY ? 0.0f : expf(-a.stats[2 * row + 1]);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float f[VEC];
            Tr::unpack(raw[n], f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) e[n * VEC + i] = f[i];
        }
    }
    const float first = m, m0 = FWD ? finite_max(m) : row_m;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) {
        e[i] = ex2((e[i] - m0) * c2);
        if (FWD) sum += e[i];
    }
    if constexpr (FWD) {
        for (uint32_t b = g0 + THREADS * NV; b < g1; b += THREADS * NV) {
            uint4 more[NV];
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const uint32_t slot = b + tid + n * THREADS;
                more[n] = slot < g1 ? load(slot) : make_uint4(low, low, low, low);
            }
            hold_batch(more);
            float bm = m, f[VEC];
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                Tr::unpack(more[n], f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) bm = fmaxf(bm, f[i]);
            }
            const float to = finite_max(bm);
            sum *= ex2((m - to) * c2);       // a thread without anything yet: 0 * 2^-inf
            m = bm;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                Tr::unpack(more[n], f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum += ex2((f[i] - to) * c2);
            }
        }
    }

    // the CTA's maxima
    {
        const float wt = warp_max(tm), wm = FWD ? warp_max(m) : 0.0f;
        if (lane == 0) {
            red[0][warp] = wt;
            red[1][warp] = wm;
        }
    }
    __syncthreads();
    float tmax = -INFINITY, cmax = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        tmax = fmaxf(tmax, red[0][w]);
        if (FWD) cmax = fmaxf(cmax, red[1][w]);
    }
    const float t0 = finite_max(tmax), cm = FWD ? finite_max(cmax) : row_m;
    // sums: the teacher's normaliser and sum e (t - tmax) / T; the CTA's part of the row
    float ts = 0.0f, tu = 0.0f, dot = 0.0f, own = 0.0f;
    for (uint32_t k = tid; k < a.kpad; k += THREADS) {
        const float u = (e_s[k] - t0) / a.temperature;
        const int id = id_s[k];
        const float w = id == -1 ? 0.0f : expf(u);
        e_s[k] = w;
        ts += w;
        if (FWD && w != 0.0f) {
            tu += w * u;
            if (id >= 0) {
                dot += w * (z_s[k] - cm);
                own += w;
            }
        }
    }
    {
        const float v0 = warp_sum(ts);
        float v1 = 0, v2 = 0, v3 = 0, v4 = 0;
        if constexpr (FWD) {
            v1 = warp_sum(tu);
            v2 = warp_sum(dot);
            v3 = warp_sum(own);
            v4 = warp_sum(sum * ex2((m - cm) * c2));
        }
        if (lane == 0) {
            red[2][warp] = v0;
            if constexpr (FWD) {
                red[3][warp] = v1;
                red[4][warp] = v2;
                red[5][warp] = v3;
                red[6][warp] = v4;
            }
        }
    }
    __syncthreads();
    if constexpr (FWD) {
        if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // every CTA of the row has begun
        if (warp == 0) {
            Part v = {cmax, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                v.dot += red[4][w];
                v.own += red[5][w];
                v.s += red[6][w];
            }
            if (lane < int(C)) {
                uint32_t at;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(uint32_t(__cvta_generic_to_shared(&parts[q]))), "r"(lane));
                asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.m), "f"(v.s), "f"(v.dot), "f"(v.own) : "memory");
            }
            __syncwarp();
        }
        if (C > 1) {
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        } else {
            __syncthreads();
        }
    }
    float tsum = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) tsum += red[2][w];
    const bool taught = tmax != -INFINITY;      // the row has a teacher
    float mx = -INFINITY, total = 0.0f;
    if constexpr (FWD) {
        for (uint32_t c = 0; c < C; ++c) mx = fmaxf(mx, parts[c].x);
        row_m = finite_max(mx);
        for (uint32_t c = 0; c < C; ++c) total += parts[c].y * ex2((parts[c].x - row_m) * c2);
        inv = total == 0.0f ? 0.0f : 1.0f / total;   // a row of nothing but -inf: p = 0
        if (q == 0 && tid == 0) {
            const float ls = logf(total);
            float d = 0.0f, u = 0.0f;
            for (uint32_t c = 0; c < C; ++c)
                if (parts[c].w != 0.0f) d += parts[c].z + parts[c].w * (finite_max(parts[c].x) - row_m);
            for (int w = 0; w < WARPS; ++w) u += red[3][w];
            float loss = 0.0f;
            if (taught) {
                if (total == 0.0f) loss = INFINITY;
                else loss = a.temperature * a.temperature * ((u / tsum - logf(tsum)) - (d / a.temperature / tsum - ls));
            }
            a.loss[row] = loss;
            if (a.stats) {
                a.stats[2 * row] = mx;
                a.stats[2 * row + 1] = ls;
            }
        }
    }
    if constexpr (BWD) {
        const float factor = (a.weight ? a.weight[row] : 1.0f) * a.temperature;
        const float scale = FWD ? inv * ex2((first - row_m) * c2) : inv;
        auto store = [&](uint32_t slot, const float (&g)[VEC]) {
            const uint32_t r = rank_of_slot(s, slot), w = shard_width(s, r);
            store_group<T>(shard_row<T>(s.out[r], s.ld, row, w), in_row(r), slot - r * s.nv, Tr::pack(g), row_ok, s.status, kSiteDistill);
        };
        for (uint32_t b = g0 + THREADS * NV; b < g1; b += THREADS * NV) {
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const uint32_t slot = b + tid + n * THREADS;
                if (slot >= g1) break;
                float f[VEC];
                Tr::unpack(load(slot), f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[i] = taught ? ex2((f[i] - row_m) * c2) * inv * factor : 0.0f;
                store(slot, f);
            }
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const uint32_t slot = g0 + tid + n * THREADS;
            if (slot >= g1) break;
            float f[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = taught ? e[n * VEC + i] * scale * factor : 0.0f;
            store(slot, f);
        }
        __syncthreads();
        if (taught) {
            for (uint32_t k = tid; k < a.k; k += THREADS) {
                const int id = id_s[k];
                if (id < 0) continue;
                float w = 0.0f;
                bool mine = true;
                for (uint32_t j = 0; j < a.kpad; j += 4) {
                    const int4 o = *reinterpret_cast<const int4 *>(&id_s[j]);
                    if (o.x == id) { w += e_s[j]; mine = mine && j >= k; }
                    if (o.y == id) { w += e_s[j + 1]; mine = mine && j + 1 >= k; }
                    if (o.z == id) { w += e_s[j + 2]; mine = mine && j + 2 >= k; }
                    if (o.w == id) { w += e_s[j + 3]; mine = mine && j + 3 >= k; }
                }
                if (!mine) continue;
                const float p = ex2((z_s[k] - row_m) * c2) * inv;
                const uint32_t r = rank_of_token(s, uint32_t(id));
                const ShardRow out = shard_row<T>(s.out[r], s.ld, row, shard_width(s, r));
                if (in_bounds(row_ok, s.status, kSiteDistill, id))
                    Tr::store1(reinterpret_cast<void *>(out.base), uint64_t(id) - shard_begin(s, r) + out.shift, (p - w / tsum) * factor);
            }
        }
    }
}

template <typename T, int PM, int PASS, int THREADS, int NV>
static cudaError_t distill_launch(const Launch &L, DistillArgs<PM> &a, uint32_t cluster, LaunchInfo *info)
{
    a.cluster = cluster;
    if (a.s.rows * cluster > 0x7fffffffull) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.s.rows * cluster));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = size_t(a.kpad) * 12;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (PASS & CCL_PASS_FORWARD) && cluster > 1 ? 2 : 1;
    cudaError_t err = cudaLaunchKernelEx(&cfg, distill_kernel<T, PM, PASS, THREADS, NV>, a);
    if (err != cudaSuccess) return err;
    info->kernel = "distill_topk";
    info->grid = int(cfg.gridDim.x);
    info->block = THREADS;
    info->smem = cfg.dynamicSmemBytes;
    info->kernels = 1;
    return cudaGetLastError();
}

template <typename T, int PM, int PASS>
static cudaError_t distill_shape(const Launch &L, const DistillLaunch &N, LaunchInfo *info)
{
    constexpr int NV = 32 / Traits<T>::VEC;   // 32 elements a thread
    DistillArgs<PM> a;
    fill_shards(&a.s, L, N.rows, N.vocab, N.ld);
    a.ids = N.ids;
    a.teacher = N.teacher;
    a.weight = N.weight;
    a.loss = N.loss;
    a.stats = N.stats;
    a.temperature = N.temperature;
    a.to_log2 = float(1.4426950408889634 / double(N.temperature));
    a.k = N.k;
    a.kpad = (N.k + 3) / 4 * 4;
    a.teacher_dtype = N.teacher_dtype;
    a.total = a.s.p * a.s.nv;
    const uint32_t per = 512 * NV;
    uint32_t C = (a.total + per - 1) / per;
    if (N.rows * C < uint64_t(L.num_sms)) {
        C = (a.total + 127) / 128;
        return distill_launch<T, PM, PASS, 128, NV>(L, a, C < 1 ? 1 : C > kDistillMaxCluster ? kDistillMaxCluster : C, info);
    }
    return distill_launch<T, PM, PASS, 512, NV>(L, a, C < 1 ? 1 : C > kDistillMaxCluster ? kDistillMaxCluster : C, info);
}

template <typename T, int PM>
static cudaError_t distill_pass(const Launch &L, const DistillLaunch &N, LaunchInfo *info)
{
    switch (N.pass) {
    case CCL_PASS_FORWARD: return distill_shape<T, PM, CCL_PASS_FORWARD>(L, N, info);
    case CCL_PASS_BACKWARD: return distill_shape<T, PM, CCL_PASS_BACKWARD>(L, N, info);
    default: return distill_shape<T, PM, CCL_PASS_BOTH>(L, N, info);
    }
}

template <typename T>
static cudaError_t distill_dtype(const Launch &L, const DistillLaunch &N, LaunchInfo *info)
{
    return L.p == 1 ? distill_pass<T, 1>(L, N, info) : L.p <= 8 ? distill_pass<T, 8>(L, N, info)
                                                                : distill_pass<T, kMaxRanks>(L, N, info);
}

cudaError_t launch_distill(const Launch &L, const DistillLaunch &N, LaunchInfo *info)
{
    switch (L.dtype) {
    case DT_F32: return distill_dtype<F32>(L, N, info);
    case DT_F16: return distill_dtype<F16>(L, N, info);
    case DT_BF16: return distill_dtype<BF16>(L, N, info);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace ccl
