// Distillation from a teacher's top K logits, the student's vocabulary split
// over the ranks: the loss, its gradient, or both in one pass.
//
// Per row, with q = softmax(t / T) over the row's valid teacher entries and
// p = softmax(z / T) over the student's vocabulary:
//   loss = T^2 sum_k q_k (log q_k - log p_{id_k})
//   dz_v = w T (p_v - sum over the k with id_k = v of q_k)
// A cluster of C CTAs takes a row.  Up to eight ranks, a CTA takes one of
// `parts` parts of one rank's shard; beyond, `teams` teams of its warps take
// one shard each.  Every thread reads its 16-byte groups once and keeps the
// first NV of them in registers as they are (16-bit types: two elements per
// register), takes the exponentials against its own maximum, and after the
// exchange of (max, sum, the teacher's share of the loss) between the CTAs
// takes them again against the row's maximum and stores the gradient: the
// logits are read once and the gradient is written once, 2 R V s bytes.
// Keeping the exponentials instead would take twice the registers and halve
// the CTAs per SM; exponentials are the cheaper of the two.  Groups past the
// first NV per thread are read a second time.  The teacher's entries are then
// put right one by one: after the CTA's barrier, the thread of an entry's
// first occurrence stores the gradient of that token with the teacher's share
// taken off.
//
// The CTAs of a row exchange their sums by writing them into one another's
// shared memory before the cluster's hardware barrier; every CTA adds the
// same C values in the same order, so all parts of a row use the same bits.
// Differences z - m are formed before the scaling by 1 / T, so that masks of
// the type's lowest value do not turn into inf - inf.
#include "logits.cuh"

namespace ccl {

constexpr int kDistillMaxCluster = 8;
constexpr int kDistillMaxThreads = 512;

template <int PM>
struct DistillArgs {
    Shards<PM> s;
    const int32_t *ids;
    const void *teacher;
    const float *weight;
    float *loss;
    float *stats;
    float temperature;
    float to_log2;        // log2(e) / T
    uint32_t k, kpad;
    uint32_t ctas;        // per row
    uint32_t parts;       // parts of a shard (teams == 1), else 1
    uint32_t teams;       // shards per CTA
    uint32_t team;        // threads of a team
    FastDiv by_ctas, by_parts, by_teams;
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

__device__ __forceinline__ float load_any(const void *p, int dtype, uint64_t i)
{
    return dtype == DT_F32 ? Traits<F32>::load1(p, i) : dtype == DT_F16 ? Traits<F16>::load1(p, i) : Traits<BF16>::load1(p, i);
}

template <typename T, int PM, int PASS, int NV, int MIN_CTAS>
__global__ void __launch_bounds__(kDistillMaxThreads, MIN_CTAS) distill_kernel(const __grid_constant__ DistillArgs<PM> a)
{
    using Tr = Traits<T>;
    using Gr = Group<T>;
    constexpr int VEC = Tr::VEC, PAIRS = Gr::PAIRS, MAX_WARPS = kDistillMaxThreads / 32;
    constexpr bool FWD = PASS & CCL_PASS_FORWARD, BWD = PASS & CCL_PASS_BACKWARD;
    extern __shared__ uint4 smem4[];
    int *id_s = reinterpret_cast<int *>(smem4);                    // ids, negative where not in this CTA's columns
    float *e_s = reinterpret_cast<float *>(id_s + a.kpad);         // exp((t - tmax) / T)
    float *z_s = e_s + a.kpad;                                     // the student's logits at the ids in these columns
    __shared__ float red[7][MAX_WARPS];
    __shared__ float4 parts[kDistillMaxCluster];                   // max, sum, teacher's dot, teacher's weight of a CTA
    const Shards<PM> &s = a.s;
    const uint32_t row32 = div_by(blockIdx.x, a.by_ctas), q = blockIdx.x - row32 * a.ctas;
    const uint64_t row = row32;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int threads = blockDim.x, warps = threads / 32;
    if (FWD && a.ctas > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    grid_dependency_wait();
    grid_dependents_launch();

    // this team's shard and part
    uint32_t r, part = 0, tt = tid;
    if (a.teams == 1) {
        r = div_by(q, a.by_parts);
        part = q - r * a.parts;
    } else {
        const uint32_t team = tid / a.team;
        r = q * a.teams + team;
        tt = tid - team * a.team;
        if (r >= s.p || team >= a.teams) r = s.p;
    }
    const bool here = r < s.p && in_bounds(row < s.rows, s.status, kSiteDistill, row);
    const uint32_t rr = here ? r : 0;
    const ShardRow<T> in(s.in[rr], s.ld, row, here ? shard_width(s, rr) : 0);
    const uint32_t whole = in.end - in.first;
    const uint32_t j0 = in.first + uint32_t(uint64_t(whole) * part / a.parts), j1 = in.first + uint32_t(uint64_t(whole) * (part + 1) / a.parts);
    const uint32_t step = a.teams == 1 ? threads : a.team;
    const int edge = in.edge(tt, part == 0, part + 1 == a.parts);

    // an id first: what it leads to comes a whole latency later
    int my_id = tid < a.k ? a.ids[row * a.k + tid] : -1;
    uint4 raw[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const uint32_t j = j0 + tt + n * step;
        raw[n] = j < j1 ? ld_coherent_v4(in.group(j)) : lowest_group<T>();
    }
    const float edge_z = edge >= 0 ? in.column(edge) : -INFINITY;

    // the teacher's entries
    float tm = -INFINITY;
    for (uint32_t k = tid; k < a.kpad; k += threads) {
        int id = k == uint32_t(tid) ? my_id : k < a.k ? a.ids[row * a.k + k] : -1;
        float t = -INFINITY, z = 0.0f;
        if (uint32_t(id) < s.vocab) {
            t = load_any(a.teacher, a.teacher_dtype, row * a.k + k);
            const uint32_t ir = rank_of_token(s, uint32_t(id)), c = uint32_t(id) - shard_begin(s, ir);
            bool mine;
            if (a.teams == 1) {
                const uint32_t lo = part == 0 ? 0u : in.head() + (j0 - in.first) * VEC;
                const uint32_t hi = part + 1 == a.parts ? in.width : in.head() + (j1 - in.first) * VEC;
                mine = ir == r && c >= lo && c < hi;
            } else {
                mine = div_by(ir, a.by_teams) == q;
            }
            if (mine) z = ShardRow<T>(s.in[ir], s.ld, row, shard_width(s, ir)).column(c);
            else id |= int(0x80000000u);     // another CTA's: only its weight counts here
        } else {
            id = -1;
        }
        id_s[k] = id;
        e_s[k] = t;
        z_s[k] = z;
        tm = fmaxf(tm, t);
    }

    // this thread's maximum and sum
    hold_batch(raw);
    const float c2 = a.to_log2;
    const Pair cc = {c2, c2};
    float m = -INFINITY, sum = 0.0f;
    float row_m = 0.0f, inv = 0.0f;
    if constexpr (FWD) {
        typename Gr::Max gm = Gr::lowest();
#pragma unroll
        for (int n = 0; n < NV; ++n) gm = Gr::max(gm, raw[n]);
        m = fmaxf(Gr::value(gm), edge_z);
        float to = finite_max(m);
        Pair acc = {ex2((edge_z - to) * c2), 0.0f};
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) acc = acc + ex2((Gr::pair(raw[n], i) + Pair{-to, -to}) * cc);
        sum = acc.x + acc.y;
        for (uint32_t j = j0 + tt + NV * step; j < j1; j += 4 * step) {
            uint4 more[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) more[n] = j + n * step < j1 ? ld_coherent_v4(in.group(j + n * step)) : lowest_group<T>();
            hold_batch(more);
            gm = Gr::lowest();
#pragma unroll
            for (int n = 0; n < 4; ++n) gm = Gr::max(gm, more[n]);
            const float bm = fmaxf(m, Gr::value(gm));
            to = finite_max(bm);
            acc = {sum * ex2((m - to) * c2), 0.0f};       // a thread without anything yet: 0 * 2^-inf
            m = bm;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) acc = acc + ex2((Gr::pair(more[n], i) + Pair{-to, -to}) * cc);
            sum = acc.x + acc.y;
        }
    } else {
        row_m = a.stats[2 * row];
        inv = row_m == -INFINITY ? 0.0f : expf(-a.stats[2 * row + 1]);
        row_m = finite_max(row_m);
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
    const float tmax = warp_max(lane < warps ? red[0][lane] : -INFINITY);
    const float cmax = FWD ? warp_max(lane < warps ? red[1][lane] : -INFINITY) : 0.0f;
    const bool taught = tmax != -INFINITY;      // the row has a teacher
    const float t0 = finite_max(tmax), cm = finite_max(cmax);
    // sums: the teacher's normaliser and sum e (t - tmax) / T; the CTA's part of the row
    float ts = 0.0f, tu = 0.0f, dot = 0.0f, own = 0.0f;
    for (uint32_t k = tid; k < a.kpad; k += threads) {
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
        const bool has = warp * 32 < int(a.kpad);   // only the first warps hold entries
        const float v0 = has ? warp_sum(ts) : 0.0f;
        float v1 = 0.0f, v2 = 0.0f, v3 = 0.0f, v4 = 0.0f;
        if constexpr (FWD) {
            if (has) {
                v1 = warp_sum(tu);
                v2 = warp_sum(dot);
                v3 = warp_sum(own);
            }
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
    const float tsum = warp_sum(lane < warps ? red[2][lane] : 0.0f);
    if constexpr (FWD) {
        if (a.ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // every CTA of the row has begun
        if (warp == 0) {
            const float vd = warp_sum(lane < warps ? red[4][lane] : 0.0f);
            const float vo = warp_sum(lane < warps ? red[5][lane] : 0.0f);
            const float vs = warp_sum(lane < warps ? red[6][lane] : 0.0f);
            if (lane < int(a.ctas)) {
                uint32_t at;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(uint32_t(__cvta_generic_to_shared(&parts[q]))), "r"(lane));
                asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(cmax), "f"(vs), "f"(vd), "f"(vo) : "memory");
            }
            __syncwarp();
        }
        if (a.ctas > 1) {
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        } else {
            __syncthreads();
        }
        const float4 mine = lane < int(a.ctas) ? parts[lane] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
        const float mx = warp_max(mine.x);
        row_m = finite_max(mx);
        const float total = warp_sum(mine.y * ex2((mine.x - row_m) * c2));
        inv = total == 0.0f ? 0.0f : 1.0f / total;   // a row of nothing but -inf: p = 0
        if (q == 0 && warp == 0) {
            const float d = warp_sum(mine.w != 0.0f ? mine.z + mine.w * (finite_max(mine.x) - row_m) : 0.0f);
            const float u = warp_sum(lane < warps ? red[3][lane] : 0.0f);
            if (lane == 0) {
                const float ls = logf(total);
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
    }
    if constexpr (BWD) {
        const float factor = (a.weight ? a.weight[row] : 1.0f) * a.temperature;
        const ShardRow<T> out(s.out[rr], s.ld, row, in.width);
        const float g = inv * factor;
        const Pair gg = {g, g}, off = {-row_m, -row_m};
        auto gradient = [&](const uint4 &v) -> uint4 {
            if (!taught) return make_uint4(0, 0, 0, 0);
            Pair p[PAIRS];
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) p[i] = ex2((Gr::pair(v, i) + off) * cc) * gg;
            return Gr::pack(p);
        };
        hold_batch(raw);    // the groups stay packed: without this the compiler keeps the unpacked values of the first pass
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const uint32_t j = j0 + tt + n * step;
            if (j < j1) store_group<T>(out, in, j, gradient(raw[n]));
        }
        for (uint32_t j = j0 + tt + NV * step; j < j1; j += step) store_group<T>(out, in, j, gradient(ld_coherent_v4(in.group(j))));
        if (edge >= 0) out.set_column(edge, taught ? ex2((edge_z - row_m) * c2) * g : 0.0f);
        __syncthreads();
        if (taught) {
            for (uint32_t k = tid; k < a.k; k += threads) {
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
                const uint32_t ir = rank_of_token(s, uint32_t(id));
                ShardRow<T>(s.out[ir], s.ld, row, shard_width(s, ir))
                    .set_column(uint32_t(id) - shard_begin(s, ir), (ex2((z_s[k] - row_m) * c2) * inv - w / tsum) * factor);
            }
        }
    }
}

template <typename T, int PM, int PASS, int NV, int MIN_CTAS>
static cudaError_t distill_launch(const Launch &L, DistillArgs<PM> &a, uint32_t need, LaunchInfo *info)
{
    // threads enough for the need of a CTA, in whole warps per team
    const uint32_t per_team = (need + NV - 1) / NV, most = kDistillMaxThreads / a.teams;
    a.team = (per_team < most ? per_team : most) / 32 * 32;
    if (a.team < per_team && a.team + 32 <= most) a.team += 32;
    if (a.team < 32) a.team = 32;
    const uint32_t threads = a.team * a.teams;
    if (a.s.rows * a.ctas > 0x7fffffffull) return cudaErrorInvalidValue;
    a.by_ctas = fast_div(a.ctas);
    a.by_parts = fast_div(a.parts);
    a.by_teams = fast_div(a.teams);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.s.rows * a.ctas));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = size_t(a.kpad) * 12;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (PASS & CCL_PASS_FORWARD) && a.ctas > 1 ? 2 : 1;
    cudaError_t err = cudaLaunchKernelEx(&cfg, distill_kernel<T, PM, PASS, NV, MIN_CTAS>, a);
    if (err != cudaSuccess) return err;
    info->kernel = "distill_topk";
    info->grid = int(cfg.gridDim.x);
    info->block = int(threads);
    info->smem = cfg.dynamicSmemBytes;
    info->kernels = 1;
    return cudaGetLastError();
}

template <typename T, int PM, int PASS>
static cudaError_t distill_shape(const Launch &L, const DistillLaunch &N, LaunchInfo *info)
{
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
    const uint32_t p = a.s.p, groups = widest_groups<T>(a.s);
    a.teams = (p + kDistillMaxCluster - 1) / kDistillMaxCluster;
    a.parts = 1;
    uint32_t need = groups;            // groups a team takes
    if (a.teams == 1) {
        // parts: few enough groups a CTA that four per thread hold them, and
        // CTAs enough for every SM
        const uint32_t most = PASS == CCL_PASS_BACKWARD ? 64 : kDistillMaxCluster / p, want = 4 * kDistillMaxThreads;
        while (a.parts < most && ((groups + a.parts - 1) / a.parts > want ||
                                  (N.rows * p * a.parts < 2 * uint64_t(L.num_sms) && (groups + a.parts - 1) / a.parts > 128)))
            ++a.parts;
        need = (groups + a.parts - 1) / a.parts;
    }
    a.ctas = a.teams == 1 ? p * a.parts : (p + a.teams - 1) / a.teams;
    const uint32_t full = need * a.teams;
    if (full <= 2 * kDistillMaxThreads) return distill_launch<T, PM, PASS, 2, 3>(L, a, need, info);
    if (PASS != CCL_PASS_BOTH || full <= 4 * kDistillMaxThreads) return distill_launch<T, PM, PASS, 4, 3>(L, a, need, info);
    return distill_launch<T, PM, PASS, 8, 2>(L, a, need, info);
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
    return L.p <= kDistillMaxCluster ? distill_pass<T, kDistillMaxCluster>(L, N, info) : distill_pass<T, kMaxRanks>(L, N, info);
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
