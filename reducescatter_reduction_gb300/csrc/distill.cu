// Distillation from a teacher's top K logits, the student's vocabulary split
// over the ranks: the loss, its gradient, or both in one pass.
//
// Per row, with q = softmax(t / T) over the row's valid teacher entries and
// p = softmax(z / T) over the student's vocabulary:
//   loss = T^2 sum_k q_k (log q_k - log p_{id_k})
//   dz_v = w T (p_v - sum over the k with id_k = v of q_k)
//
// A row is cut into Q pieces, each a part of one rank's shard or several
// whole shards (small ones, and beyond 16 ranks; for the loss alone also parts
// of neighbours), and a persistent CTA takes one piece of one
// row after another.  Where the loss is computed the Q CTAs of a row form a
// cluster and go through the rows together.  Ten or eleven warps, tied
// together by mbarriers alone:
//
//   warp 8 (loads and patches)  brings the 16-byte groups of the piece of a
//                               coming row into a stage of shared memory with
//                               one bulk copy per shard, its edge elements and
//                               where they go beside it, S stages ahead
//   warp 9, 10 (teacher)        softmax of the row's teacher entries, the
//                               student's logits at those in the piece, and
//                               their share of the loss
//   warps 0-7 (consumers)       take a stage into registers and free it;
//                               exponentials against the thread's own maximum,
//                               (max, sum) per warp to every CTA of the row;
//                               from all of them the row's maximum and sum;
//                               scale the exponentials into the gradient and
//                               store it
//   warp 8 again                stores the gradient at the teacher's tokens
//                               once the consumers' stores are out, each
//                               token by its first entry
//
// So the logits are read once, the gradient is written once, each element
// costs one exponential, and while a row's sums travel the next rows' loads
// are in flight.  What the CTAs tell one another goes into
// slots with st.async and is counted by the receiver's mbarrier; every CTA
// adds the same values in the same order, so all pieces of a row use the same
// bits.  There are four slots, and a sender's sums for row k leave only after
// all of row k - 2 has reached it: by then every CTA has sent its sums of row
// k - 2, so it is done with the sums of row k - 4, which had the slot before
// (its teacher's warp sends row k - 2 only after the loss of row k - 4; where
// there are two, rows k, k - 2 and k - 4 are the same one's).
// (For the loss alone the consumers see a row complete two rows later.)
//
// A piece beyond 2048 groups (vocabularies above 262144 16-bit or 131072
// 32-bit columns on up to 16 ranks a power of two) is taken in chunks: the
// sums go through them once, the gradient reads them a second time.
//
// Differences z - m are formed before the scaling by 1 / T, so that masks of
// the type's lowest value do not turn into inf - inf.
//
// Measured (graph replay): loss and gradient, 4096 x 131072 bf16 on 8 ranks,
// 64 entries: 410-430 us (5.0-5.2 TB/s), bound by the teacher's warp and by
// the exchange's latency (8 entries: 386, 128: 665, 256: 620); 700 x 100003
// bf16 on 3, whose pieces fill two thirds of a stage: 87-93 us.  The loss
// alone, 2048 x 65536 f16: 53 us (5.1 TB/s); the gradient alone, f32: 179 us
// (6.0 TB/s).
//
// Every wait is bounded by the communicator's wait limit; one that gives up
// records itself in the status block, and the CTA leaves its loops, waits
// (bounded) for its copies in flight and for the other CTAs of the row, and
// returns.
#include "async.cuh"
#include "logits.cuh"

namespace ccl {

constexpr int kDistillConsumers = 256;
constexpr int kDistillWarps = kDistillConsumers / 32;
// One teacher's warp, or two that take the rows in turn.  One against two, us:
// 4096 x 131072 bf16 with 256 entries, loss and gradient 1026 and 632, the
// gradient alone 671 and 467.  With 128 entries it is this way and that: 664
// and 628, the gradient alone 374 and 383; 700 x 100003 bf16 113 and 123; 16 x
// 32000 f32 5.3 and 5.8; the gradient of 2048 x 65536 f32 177 and 165.  So two
// from 129 entries on, with three in a lane's registers, as two have fewer
// registers each.
template <int HELD>
constexpr int kDistillTeachers = HELD == 3 ? 2 : 1;
template <int HELD>
constexpr int kDistillThreads = kDistillConsumers + 32 + 32 * kDistillTeachers<HELD>;
constexpr int kDistillGroups = 8;                                      // groups a consumer takes of a stage
constexpr uint32_t kDistillStage = kDistillConsumers * kDistillGroups; // groups of a stage
constexpr uint32_t kDistillStageBytes = kDistillStage * 16;

// What a pass is built for.  The loss alone keeps no exponentials, so an SM
// holds three CTAs of it instead of two (of two stages instead of three), in
// clusters of up to eight: beyond, its pieces come in chunks, which cost it
// less than clusters of sixteen (2048 x 262144 bf16 on 8 ranks: 194 against
// 229 us; 2048 x 65536 f16 on 16: 116 against 235).  Three CTAs against two:
// 2048 x 65536 f16, 62 against 75 us at the time.
template <int PASS>
struct DistillShape {
    static constexpr bool loss_alone = PASS == CCL_PASS_FORWARD;
    static constexpr int ctas = loss_alone ? 3 : 2;              // per SM
    static constexpr uint32_t stages = loss_alone ? 2 : 3;
    static constexpr int cluster = loss_alone ? 8 : 16;          // pieces of a row
    static constexpr int segments = kMaxRanks / cluster;         // shards of a piece
    static constexpr size_t smem = (loss_alone ? 75 : 113) * 1024;   // of a CTA, a kilobyte of the system's included
};

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
    uint32_t share;       // the entries of a piece for the loss alone: those of all pieces make a row's
    uint32_t pieces;      // per row
    uint32_t parts;       // parts of a shard (one shard a piece), else 1
    uint32_t segments;    // shards of a piece, at most
    uint32_t span;        // the loss alone, if not 0: a piece's groups, counted as if every shard had `groups`
    uint32_t groups;      // of the widest shard
    uint32_t chunks;      // of a piece
    uint32_t stages;
    uint32_t items;       // rows * pieces
    FastDiv by_pieces, by_parts, by_segments, by_groups;
    int teacher_dtype;
    int edges;            // some row begins or ends between 16-byte boundaries
    long long wait_ns;
    int stall_test;       // 1: the second load of every CTA is withheld, so that a wait runs out (tests)
};

// Where a stage's groups and edge elements go.
template <int PASS>
struct DistillDesc {
    static constexpr int SEGS = DistillShape<PASS>::segments;
    struct Segment {
        uint64_t out;          // address of the output of its first group
        uint32_t first;        // its first group in the stage
        uint32_t aligned;      // the output's groups lie on 16-byte boundaries too
    } seg[SEGS];
    uint64_t edge_out[SEGS * 16];   // address of an edge element's output, 0: no such element
    float edge[SEGS * 16];
    uint32_t groups;
};

// What reaches a CTA from the CTAs of its row.  The teacher's part of the
// loss is a sum over its entries, so for the loss alone each piece takes a
// share of the entries, wherever in the vocabulary they are, against a maximum
// of its own; where a gradient follows, each goes through all of them for the
// weights of those in its columns.
template <int PASS>
struct DistillSums {
    float2 warp[DistillShape<PASS>::cluster][kDistillWarps];   // max, sum
    // reference, sum e (z - reference) / 1024 and sum e over the piece's entries, sum e over all of them (the loss alone: the
    // maximum t that e is against) | sum e (t - maximum) / T, the row's weight
    float4 teacher[DistillShape<PASS>::cluster][2];
};
constexpr int kDistillSlots = 4, kDistillLag = 2;
constexpr uint32_t kDistillSumBytes = kDistillWarps * 8 + 32;   // from one CTA

template <int PASS>
struct DistillShared {
    DistillSums<PASS> sums[kDistillSlots];
    DistillDesc<PASS> desc[DistillShape<PASS>::stages + 1];
    uint64_t full[DistillShape<PASS>::stages], empty[DistillShape<PASS>::stages];
    uint64_t sums_in[kDistillSlots], taught[2], taught_free[2], stored[2];
    uint32_t entries[2];                              // the piece's teacher entries
    float teacher_sum[2];
    float weight[2], row_max[2], row_log_sum[2];      // of the row (the latter two for a gradient alone)
    float used_max[2], used_inv[2];                   // what the consumers scaled by
    int dead;
};

// The maximum of a warp; a NaN is passed over.
__device__ __forceinline__ float warp_max(float v)
{
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
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

__device__ __forceinline__ uint32_t remote(uint32_t local, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ void send2(uint32_t at, uint32_t bar, float x, float y)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(at), "r"(__float_as_uint(x)),
                 "r"(__float_as_uint(y)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void send4(uint32_t at, uint32_t bar, float4 v)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
                 "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)), "r"(__float_as_uint(v.w)), "r"(bar)
                 : "memory");
}

// Values that other CTAs wrote: cluster scope.
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits for a phase, bounded; false if the wait, or any wait of this CTA, gave up.
template <int PM, int PASS>
__device__ __forceinline__ bool distill_wait(const DistillArgs<PM> &a, DistillShared<PASS> &sh, uint64_t *barrier, uint32_t parity, unsigned code,
                                             uint32_t item)
{
    const uint32_t bar = smem_addr(barrier);
    if (try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    volatile int *dead = &sh.dead;
    while (!try_wait_cluster(bar, parity)) {
        if (*dead) return false;
        if (global_ns() - t0 > uint64_t(a.wait_ns)) {
            if (atomicCAS(&a.s.status[0], 0u, code) == 0u) {
                a.s.status[1] = blockIdx.x;
                a.s.status[2] = item;
                a.s.status[3] = threadIdx.x;
            }
            *dead = 1;
            return false;
        }
    }
    return true;
}

// Waits for all of the sums of this CTA's k-th row.
template <int PM, int PASS>
__device__ __forceinline__ bool wait_sums(const DistillArgs<PM> &a, DistillShared<PASS> &sh, uint32_t k, unsigned code, uint32_t item)
{
    return __all_sync(0xffffffffu, distill_wait(a, sh, &sh.sums_in[k % kDistillSlots], (k / kDistillSlots) & 1, code, item));
}

// What piece q of a row takes of shard `rank`, its segment seg (rank >= p: there is none).
template <typename T, int PM, int PASS>
struct Piece {
    uint32_t rank;
    uint32_t lo, hi;       // of several shards: its groups of this one
    uint32_t part;         // of one shard
    bool head, tail;       // the shard's first and last columns are of this piece
    uint32_t j0, j1;       // its groups

    __device__ __forceinline__ Piece(const DistillArgs<PM> &a, uint32_t q, uint32_t seg)
    {
        part = lo = 0;
        hi = 0xffffffffu;
        head = tail = true;
        if (a.segments == 1) {
            rank = div_by(q, a.by_parts);
            part = q - rank * a.parts;
            head = part == 0;
            tail = part + 1 == a.parts;
        } else if (PASS != CCL_PASS_FORWARD || !a.span) {
            rank = q * a.segments + seg;
        } else {
            const uint32_t from = q * a.span, first = div_by(from, a.by_groups);
            rank = first + seg;
            lo = seg ? 0u : from - first * a.groups;
            const uint32_t begin = rank * a.groups, end = from + a.span;
            if (end <= begin) rank = a.s.p;
            hi = min(a.groups, end - begin);
            head = lo == 0;
            tail = hi == a.groups;
        }
    }
    __device__ __forceinline__ void cut(const DistillArgs<PM> &a, const ShardRow<T, PM> &row)
    {
        const uint32_t whole = row.end - row.first;
        if (a.segments == 1) {
            const uint32_t per = div_by(whole + a.parts - 1, a.by_parts);
            lo = per * part;
            hi = per * (part + 1);
        }
        j0 = row.first + min(whole, lo);
        j1 = row.first + min(whole, hi);
    }
};

// HELD: teacher entries of a lane in registers.  The teacher's warp bounds loss and gradient together, so it holds no
// more than the call has: 64 entries, 4096 x 131072 bf16: 423 us with two a lane, 528 with four.
template <typename T, int PM, int PASS, int HELD>
__global__ void __launch_bounds__(kDistillThreads<HELD>, DistillShape<PASS>::ctas) distill_kernel(const __grid_constant__ DistillArgs<PM> a)
{
    using Tr = Traits<T>;
    using Gr = Group<T>;
    constexpr int VEC = Tr::VEC, PAIRS = Gr::PAIRS, NG = kDistillGroups;
    constexpr bool FWD = PASS & CCL_PASS_FORWARD, BWD = PASS & CCL_PASS_BACKWARD;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ DistillShared<PASS> sh;
    const Shards<PM> &s = a.s;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t S = a.stages;
    // behind the stages: two slots of the piece's teacher entries (ids, exp((t - tmax) / T), logits), and the room of
    // the teacher's warp for what its registers do not hold
    int *id_s = reinterpret_cast<int *>(smem + size_t(S) * kDistillStageBytes);
    float *e_s = reinterpret_cast<float *>(id_s + 2 * a.kpad), *z_s = e_s + 2 * a.kpad;
    int *more = BWD ? reinterpret_cast<int *>(z_s + 2 * a.kpad) : id_s;

    if (tid == 0) {
        for (uint32_t i = 0; i < S; ++i) {
            mbar_init(smem_addr(&sh.full[i]), 1);
            mbar_init(smem_addr(&sh.empty[i]), kDistillWarps);
        }
        for (int i = 0; i < kDistillSlots; ++i) mbar_init(smem_addr(&sh.sums_in[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.taught[i]), 1);
            mbar_init(smem_addr(&sh.taught_free[i]), 1);
            mbar_init(smem_addr(&sh.stored[i]), kDistillWarps);
        }
        sh.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (FWD) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    grid_dependency_wait();
    grid_dependents_launch();

    // chunks that an item loads: a piece of several is read once for the sums and once for the gradient
    const uint32_t loads = PASS == CCL_PASS_BOTH && a.chunks > 1 ? 2 * a.chunks : a.chunks;
    const uint32_t stride = gridDim.x;
    uint32_t issued = 0;

    const float c2 = a.to_log2;
    // The row's maximum and the sum of its exponentials, from all its CTAs' sums.
    auto total_of = [&](uint32_t slot, float &mx) -> float {
        constexpr int EACH = DistillShape<PASS>::cluster * kDistillWarps / 32;
        const float2 *pairs = &sh.sums[slot].warp[0][0];
        const uint32_t n = a.pieces * kDistillWarps;
        float2 v[EACH];
        mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            v[i] = lane + 32 * i < n ? pairs[lane + 32 * i] : make_float2(-INFINITY, 0.0f);
            mx = fmaxf(mx, v[i].x);
        }
        mx = warp_max(mx);
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < EACH; ++i) total += v[i].y * ex2((v[i].x - finite_max(mx)) * c2);
        return warp_sum(total);
    };
    // The row's loss: one warp of its pieces in turn, two rows later, a consumer for the loss alone, else the teacher's.  (In the
    // consumers' or the patching warp's way it would hold up all the CTAs of the row.)
    auto finish_row = [&](uint32_t slot, uint32_t row) {
        const DistillSums<PASS> &in = sh.sums[slot];
        float mx;
        const float total = total_of(slot, mx), row_m = finite_max(mx);
        const float4 t = lane < int(a.pieces) ? in.teacher[lane][0] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float tsum, u, part = t.z;      // part: the entries' share of sum e
        if constexpr (BWD) {
            tsum = in.teacher[0][0].w;
            u = in.teacher[0][1].x;
        } else {
            // the shares' maxima and sums together
            const float top = warp_max(t.z != 0.0f ? t.w : -INFINITY), scale = t.z != 0.0f ? ex2((t.w - finite_max(top)) * c2) : 0.0f;
            u = t.z != 0.0f ? scale * (in.teacher[lane][1].x + t.z * (t.w - top) / a.temperature) : 0.0f;
            part *= scale;
            tsum = warp_sum(part);
            u = warp_sum(u);
        }
        // sum q (z - the row's maximum)
        const float dot = warp_sum(part != 0.0f ? part / tsum * (t.y / t.z * 1024.0f + (t.x - row_m)) : 0.0f);
        if (lane == 0) {
            const float ls = logf(total), heat = a.temperature;
            float loss = 0.0f;
            if (tsum != 0.0f) {
                if (total == 0.0f) loss = INFINITY;
                else loss = heat * (heat * ((u / tsum - logf(tsum)) - (dot / heat - ls)));   // heat^2 may be out of range
            }
            if (!row_held(s, row)) return;
            a.loss[row] = loss;
            if (a.stats) {
                a.stats[2 * uint64_t(row)] = mx;
                a.stats[2 * uint64_t(row) + 1] = ls;
            }
        }
    };

    if (warp == kDistillWarps) {
        // ---- loads, and the gradient at the teacher's tokens -------------
        const uint32_t count = (a.items - blockIdx.x + stride - 1) / stride;   // items of this CTA: at least one
        uint32_t item = blockIdx.x, load = 0;                                  // the next to issue
        // edge element e of the pieces of a load, as ShardRow::edge numbers them; a lane's first comes in ahead of its load
        auto edge_of = [&](uint32_t of, uint32_t part, uint32_t e, float &z, uint64_t &to) {
            const uint32_t row = div_by(of, a.by_pieces), c = part % a.chunks;
            Piece<T, PM, PASS> pe(a, of - row * a.pieces, e / (2 * VEC));
            z = -INFINITY;
            to = 0;
            if (pe.rank >= s.p) return;
            const ShardRow<T, PM> in(s, s.in[pe.rank], pe.rank, row);
            const int col = in.edge(e % (2 * VEC), pe.head && c == 0, pe.tail && c + 1 == a.chunks);
            if (col < 0) return;
            z = in.column(col);
            if (BWD) {
                const ShardRow<T, PM> out(s, s.out[pe.rank], pe.rank, row);
                to = out.base + (uint64_t(out.shift) + uint32_t(col)) * (16 / VEC);
            }
        };
        float edge_z = -INFINITY;
        uint64_t edge_to = 0;
        auto prefetch_edge = [&]() {
            if (a.edges && item < a.items && lane < int(a.segments * 2 * VEC)) edge_of(item, load, lane, edge_z, edge_to);
        };
        prefetch_edge();
        auto issue = [&]() -> bool {
            const uint32_t st = issued % S;
            if (issued >= S && !__all_sync(0xffffffffu, distill_wait(a, sh, &sh.empty[st], (issued / S - 1) & 1, 6, item))) return false;
            DistillDesc<PASS> &d = sh.desc[issued % (S + 1)];
            const uint32_t row = div_by(item, a.by_pieces), q = item - row * a.pieces, c = load % a.chunks;
            const uint32_t cap = a.segments == 1 || (PASS == CCL_PASS_FORWARD && a.span) ? kDistillStage : div_by(kDistillStage, a.by_segments);
            // lane l: segment l
            uint32_t n = 0;
            const void *from = nullptr;
            Piece<T, PM, PASS> pc(a, q, lane);
            if (lane < int(a.segments) && pc.rank < s.p) {
                const ShardRow<T, PM> in(s, s.in[pc.rank], pc.rank, row);
                pc.cut(a, in);
                const uint32_t k0 = min(pc.j0 + c * cap, pc.j1), k1 = min(k0 + cap, pc.j1);
                from = in.group(k0);
                if (k0 == k1 || in.holds(from, (k1 - k0) * 16)) n = k1 - k0;
                if (BWD) {
                    const ShardRow<T, PM> out(s, s.out[pc.rank], pc.rank, row);
                    const uintptr_t at = out.base + (uint64_t(out.shift) + k0 * VEC - in.shift) * (16 / VEC);
                    d.seg[lane].out = at;
                    d.seg[lane].aligned = at % 16 == 0;
                }
            }
            uint32_t first = 0, all = 0;
            if (a.segments == 1) all = __shfl_sync(0xffffffffu, n, 0);
            else
#pragma unroll
            for (int l = 0; l < DistillShape<PASS>::segments; ++l) {
                const uint32_t m = __shfl_sync(0xffffffffu, n, l);
                if (l < lane) first += m;
                all += m;
            }
            const bool held = a.stall_test == 1 && issued == 1;
            const uint32_t bar = smem_addr(&sh.full[st]);
            if (n && !held) bulk_load(smem_addr(smem) + st * kDistillStageBytes + first * 16, from, n * 16, bar);
            if (lane < int(a.segments)) d.seg[lane].first = first;
            if (a.edges && lane < int(a.segments * 2 * VEC)) {
                d.edge[lane] = edge_z;
                d.edge_out[lane] = edge_to;
            }
            for (uint32_t e = lane + 32; a.edges && e < a.segments * 2 * VEC; e += 32) edge_of(item, load, e, d.edge[e], d.edge_out[e]);
            if (lane == 0) d.groups = all;
            __syncwarp();
            if (lane == 0 && !held) mbar_arrive_expect_tx(bar, all * 16);
            ++issued;
            if (++load == loads) {
                load = 0;
                item += stride;
            }
            prefetch_edge();
            return true;
        };
        const uint32_t every = count * loads;
        bool ok = true;
        uint32_t row_item = blockIdx.x;
        for (uint32_t k = 0; k < count && ok; ++k, row_item += stride) {
            // all of this item's loads, and S - 1 beyond: the last of them waits for the stage before this item's last
            const uint64_t until = uint64_t(k + 1) * loads + S - 1;
            while (ok && issued < every && issued < until) ok = issue();
            if constexpr (BWD) {
                const uint32_t slot = k & 1, parity = (k >> 1) & 1;
                ok = ok && __all_sync(0xffffffffu, distill_wait(a, sh, &sh.taught[slot], parity, 7, row_item));
                if (!ok) break;
                const uint32_t row = div_by(row_item, a.by_pieces);
                // 1 / the teacher's sum, which is 1 or more: the approximate reciprocal and a step of Newton's iteration, right to
                // half an ulp.  Measured (2048 x 80768 bf16 on 8 ranks): 208 us, with a division in its place 218.
                const float tsum = sh.teacher_sum[slot], approx = __fdividef(1.0f, tsum), tinv = fmaf(fmaf(-tsum, approx, 1.0f), approx, approx);
                ok = __all_sync(0xffffffffu, distill_wait(a, sh, &sh.stored[slot], parity, 7, row_item));
                if (!ok) break;
                const float row_m = sh.used_max[slot], inv = sh.used_inv[slot];
                const float factor = sh.weight[slot] * a.temperature;
                const uint32_t n = sh.entries[slot];
                const int *ids = id_s + slot * a.kpad;
                const float *es = e_s + slot * a.kpad, *zs = z_s + slot * a.kpad;
                for (uint32_t i = lane; i < n; i += 32) {
                    const int id = ids[i];
                    float w = 0.0f;
                    bool mine = true;      // the token's first entry stores for all of them
                    for (uint32_t j = 0; j < n; j += 4) {
                        const int4 o = *reinterpret_cast<const int4 *>(&ids[j]);
                        if (o.x == id) { w += es[j]; mine = mine && j >= i; }
                        if (o.y == id) { w += es[j + 1]; mine = mine && j + 1 >= i; }
                        if (o.z == id) { w += es[j + 2]; mine = mine && j + 2 >= i; }
                        if (o.w == id) { w += es[j + 3]; mine = mine && j + 3 >= i; }
                    }
                    if (!mine) continue;
                    const uint32_t r = rank_of_token(s, uint32_t(id));
                    ShardRow<T, PM>(s, s.out[r], r, row)
                        .set_column(uint32_t(id) - shard_begin(s, r), (ex2((zs[i] - row_m) * a.to_log2) * inv - w * tinv) * factor);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.taught_free[slot]));
            }
        }
    } else if (warp > kDistillWarps) {
        // ---- the teacher's entries ---------------------------------------
        // 32 U of a row are held in registers: their ids and logits are
        // loaded two rows ahead, the student's logits at them one row ahead.
        // Any others are loaded when it is their turn and kept in shared memory.
        constexpr int U = HELD;
        constexpr uint32_t ES = 16 / VEC;
        struct Held {
            int id[U];
            float t[U], z[U];
            float w, max, log_sum;
        };
        Held coming, next, now;
        // this piece's entries of a row (the same piece of every row where the CTAs form a cluster)
        const uint32_t begin = BWD ? 0u : min((blockIdx.x % a.pieces) * a.share, a.k), share = BWD ? a.k : min(a.share, a.k - begin);
        auto held_entry = [&](uint64_t at) { return in_bounds(at < s.held * a.k, s.status, s.site, at); };
        auto fetch = [&](uint32_t item) {
            if (item >= a.items) return;
            const uint32_t row = div_by(item, a.by_pieces);
            const bool listed = row_held(s, row);
            const uint64_t at = uint64_t(row) * a.k + begin + lane;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (32 * u >= share) {
                    coming.id[u] = -1;
                    coming.t[u] = -INFINITY;
                    continue;
                }
                const bool in = lane + 32 * u < share && listed && held_entry(at + 32 * u);
                coming.id[u] = in ? a.ids[at + 32 * u] : -1;
                coming.t[u] = in ? load_any(a.teacher, a.teacher_dtype, at + 32 * u) : -INFINITY;
            }
            coming.w = BWD && a.weight && listed ? a.weight[row] : 1.0f;
            if (!FWD) {
                coming.max = listed ? a.stats[2 * uint64_t(row)] : 0.0f;
                coming.log_sum = listed ? a.stats[2 * uint64_t(row) + 1] : 0.0f;
            }
        };
        // What a piece holds: tokens [from, to), consecutive in memory from `at` on where it is of one shard.
        struct Hold {
            uint32_t row, from, count;
            uintptr_t at;
        };
        auto hold_of = [&](uint32_t item) -> Hold {
            Hold h;
            h.row = div_by(item, a.by_pieces);
            const uint32_t q = item - h.row * a.pieces;
            h.at = 0;
            if (!BWD) {
                h.from = 0;
                h.count = s.vocab;
            } else if (a.segments == 1) {
                Piece<T, PM, PASS> pc(a, q, 0);
                const ShardRow<T, PM> in(s, s.in[pc.rank], pc.rank, h.row);
                pc.cut(a, in);
                const uint32_t lo = pc.head ? 0u : in.head() + (pc.j0 - in.first) * VEC;
                const uint32_t hi = pc.tail ? in.width : in.head() + (pc.j1 - in.first) * VEC;
                h.from = shard_begin(s, pc.rank) + lo;
                h.count = hi - lo;
                h.at = in.base + uint64_t(in.shift + lo) * ES;
            } else {
                h.from = shard_begin(s, min(q * a.segments, s.p));
                h.count = shard_begin(s, min((q + 1) * a.segments, s.p)) - h.from;
            }
            return h;
        };
        // an entry outside the vocabulary: id -1; of another piece: the sign bit set, only its weight counts here
        auto place = [&](const Hold &h, int &id, float &t, float &z) {
            z = 0.0f;
            if (uint32_t(id) - h.from < h.count) {
                if (BWD && a.segments == 1) {
                    if constexpr (kBoundsCheck) {
                        const uint32_t r = rank_of_token(s, uint32_t(id));
                        if (!ShardRow<T, PM>(s, s.in[r], r, h.row).holds(reinterpret_cast<const void *>(h.at + uintptr_t(uint32_t(id) - h.from) * ES), ES)) return;
                    }
                    z = Tr::load1(reinterpret_cast<const void *>(h.at), uint32_t(id) - h.from);
                } else {
                    const uint32_t r = rank_of_token(s, uint32_t(id));
                    z = ShardRow<T, PM>(s, s.in[r], r, h.row).column(uint32_t(id) - shard_begin(s, r));
                }
            } else if (uint32_t(id) < s.vocab) {
                id |= int(0x80000000u);
            } else {
                id = -1;
                t = -INFINITY;
            }
        };
        auto place_all = [&](uint32_t item) {
            if (item >= a.items) return;
            const Hold h = hold_of(item);
            next = coming;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (32 * u < share) place(h, next.id[u], next.t[u], next.z[u]);
        };
        constexpr uint32_t TEACHERS = kDistillTeachers<HELD>;
        const uint32_t who_am_i = warp - kDistillWarps - 1, turn = TEACHERS * stride;
        int *more_id = more + 3 * who_am_i * a.kpad;
        float *more_e = reinterpret_cast<float *>(more_id + a.kpad), *more_z = more_e + a.kpad;
        uint32_t k = who_am_i;
        const uint32_t item0 = blockIdx.x + who_am_i * stride;
        fetch(item0);
        place_all(item0);
        fetch(item0 + turn);
        const float per_t = 1.0f / a.temperature;
        for (uint32_t item = item0; item < a.items; item += turn, k += TEACHERS) {
            const uint32_t slot = k & 1;
            const uint32_t row = div_by(item, a.by_pieces), q = item - row * a.pieces;
            now = next;
            place_all(item + turn);
            fetch(item + 2 * turn);
            float tm = -INFINITY, ref = -INFINITY;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                tm = fmaxf(tm, now.t[u]);
                if (now.id[u] >= 0 && now.z[u] < INFINITY) ref = fmaxf(ref, now.z[u]);
            }
            if (share > 32 * U) {
                const Hold h = hold_of(item);
                const uint64_t at = uint64_t(row) * a.k + begin;
                constexpr int M = 4;          // loads in flight
                for (uint32_t i0 = lane + 32 * U; i0 - lane < share; i0 += 32 * M) {
                    int id[M];
                    float t[M], z[M];
#pragma unroll
                    for (int u = 0; u < M; ++u) {
                        const bool in = i0 + 32 * u < share && held_entry(at + i0 + 32 * u);
                        id[u] = in ? a.ids[at + i0 + 32 * u] : -1;
                        t[u] = in ? load_any(a.teacher, a.teacher_dtype, at + i0 + 32 * u) : -INFINITY;
                    }
#pragma unroll
                    for (int u = 0; u < M; ++u) place(h, id[u], t[u], z[u]);
#pragma unroll
                    for (int u = 0; u < M; ++u) {
                        const uint32_t i = i0 + 32 * u;
                        if (i >= share) break;
                        more_id[i] = id[u];
                        more_e[i] = t[u];
                        more_z[i] = z[u];
                        tm = fmaxf(tm, t[u]);
                        if (id[u] >= 0 && z[u] < INFINITY) ref = fmaxf(ref, z[u]);
                    }
                }
            }
            tm = finite_max(warp_max(tm));
            if (FWD) ref = finite_max(warp_max(ref));
            if (BWD && k >= 2 && !__all_sync(0xffffffffu, distill_wait(a, sh, &sh.taught_free[slot], ((k >> 1) - 1) & 1, 8, item))) break;
            float ts = 0.0f, tu = 0.0f, dot = 0.0f, own = 0.0f;
            uint32_t kept = 0;
            // an entry's weight: summed up, and kept where a gradient needs it
            auto weigh = [&](int eid, float et, float ez) {
                const float u = (et - tm) * per_t;
                const float e = eid == -1 ? 0.0f : ex2((et - tm) * a.to_log2);
                ts += e;
                const bool mine = e != 0.0f && eid >= 0;
                if (FWD && e != 0.0f) tu += e * u;
                if (FWD && mine) {
                    own += e;
                    // a 1024th: at most so many entries, so masks of the lowest value do not leave fp32's range
                    dot += e * 0x1p-10f * (ez - ref);
                }
                if (BWD) {
                    const unsigned who = __ballot_sync(0xffffffffu, mine);
                    const uint32_t at = slot * a.kpad + kept + __popc(who & ((1u << lane) - 1));
                    if (mine) {
                        id_s[at] = eid;
                        e_s[at] = e;
                        z_s[at] = ez;
                    }
                    kept += __popc(who);
                }
            };
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (32 * u < share) weigh(now.id[u], now.t[u], now.z[u]);
            for (uint32_t i0 = 32 * U; i0 < share; i0 += 32) {
                const uint32_t i = i0 + lane;
                const bool in = i < share;
                weigh(in ? more_id[i] : -1, in ? more_e[i] : 0.0f, in ? more_z[i] : 0.0f);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float v0 = __shfl_xor_sync(0xffffffffu, ts, o);
                if constexpr (FWD) {
                    const float v1 = __shfl_xor_sync(0xffffffffu, tu, o), v2 = __shfl_xor_sync(0xffffffffu, dot, o),
                                v3 = __shfl_xor_sync(0xffffffffu, own, o);
                    tu += v1;
                    dot += v2;
                    own += v3;
                }
                ts += v0;
            }
            if constexpr (BWD) {
                if (kept % 4 && lane < int(4 - kept % 4)) id_s[slot * a.kpad + kept + lane] = -1;
                if (lane == 0) {
                    sh.entries[slot] = ts != 0.0f ? kept : 0u;
                    sh.teacher_sum[slot] = ts;
                    sh.weight[slot] = now.w;
                    sh.row_max[slot] = now.max;
                    sh.row_log_sum[slot] = now.log_sum;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.taught[slot]));
            }
            if constexpr (FWD) {
                if (k >= kDistillLag && !wait_sums(a, sh, k - kDistillLag, 9, item)) break;
                // (before this row's sums leave: with them the others may go on to the row that gets its slot)
                if (BWD && k >= kDistillLag && q == (k - kDistillLag) % a.pieces)
                    finish_row((k - kDistillLag) % kDistillSlots, div_by(item - kDistillLag * stride, a.by_pieces));
                const uint32_t to = k % kDistillSlots;
                if (lane == 0) mbar_arrive_expect_tx(smem_addr(&sh.sums_in[to]), a.pieces * kDistillSumBytes);
                if (lane < int(a.pieces)) {
                    const uint32_t bar = remote(smem_addr(&sh.sums_in[to]), lane), at = remote(smem_addr(&sh.sums[to].teacher[q][0]), lane);
                    send4(at, bar, make_float4(ref, dot, own, BWD ? ts : tm));
                    send4(at + 16, bar, make_float4(tu, now.w, 0.0f, 0.0f));
                }
            }
        }
        if constexpr (FWD && BWD) {
            // the last rows' losses
            const uint32_t rows = (a.items - blockIdx.x + stride - 1) / stride;
            for (uint32_t j = rows > kDistillLag ? rows - kDistillLag : 0u; j < rows; ++j) {
                const uint32_t item = blockIdx.x + j * stride, row = div_by(item, a.by_pieces);
                if (j % TEACHERS != who_am_i) continue;
                if (!wait_sums(a, sh, j, 14, item)) break;
                if (item - row * a.pieces == j % a.pieces) finish_row(j % kDistillSlots, row);
            }
        }
    } else {
        // ---- consumers ---------------------------------------------------
        const Pair cc = {c2, c2};
        const uint32_t stages_at = smem_addr(smem);
        uint32_t used = 0, k = 0;
        for (uint32_t item = blockIdx.x; item < a.items; item += stride, ++k) {
            const uint32_t slot = k & 1, parity = (k >> 1) & 1;
            const uint32_t row = div_by(item, a.by_pieces), q = item - row * a.pieces;
            // the loss alone takes a stage by halves, the others keep all of it
            constexpr int TAKE = BWD ? NG : NG / 2;
            Pair e[TAKE * PAIRS];
            float m = -INFINITY, sum = 0.0f, edge = -INFINITY;
            bool ok = true;
            const DistillDesc<PASS> *d = nullptr;
            // the next chunk's stage, once it is full
            auto arrive = [&]() {
                ok = __all_sync(0xffffffffu, distill_wait(a, sh, &sh.full[used % S], (used / S) & 1, 10, item));
                if (!ok) return;
                d = &sh.desc[used % (S + 1)];
                edge = a.edges && uint32_t(tid) < a.segments * 2 * VEC ? d->edge[tid] : -INFINITY;
            };
            // its groups from `part` on into e; the stage free again after the last
            auto take = [&](int part) -> typename Gr::Max {
                const uint32_t st = used % S, at = stages_at + st * kDistillStageBytes + tid * 16, groups = d->groups;
                typename Gr::Max gm = Gr::lowest();
#pragma unroll
                for (int n = 0; n < TAKE; ++n) {
                    const uint32_t g = (part + n) * kDistillConsumers;
                    const uint4 v = tid + g < groups ? lds_v4(at + g * 16) : lowest_group<T>();
                    gm = Gr::max(gm, v);
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) e[n * PAIRS + i] = Gr::pair(v, i);
                }
                if (part + TAKE == NG) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh.empty[st]));
                    ++used;
                }
                return gm;
            };
            // (checked build) a store of segment sg's lies in the output of its rank
            auto stores = [&](uint32_t sg, const void *to, uint32_t bytes) -> bool {
                if constexpr (!kBoundsCheck) return true;
                const Piece<T, PM, PASS> ps(a, q, sg);
                return in_bounds(ps.rank < s.p, s.status, s.site, row) && ShardRow<T, PM>(s, s.out[ps.rank], ps.rank, row).holds(to, bytes);
            };
            // stores e * g (edge: edge * g) where the chunk came from; zero for a row without a teacher
            auto put = [&](float g, bool taught) {
                const uint32_t groups = d->groups;
                const Pair gg = {taught ? g : 0.0f, taught ? g : 0.0f};
                auto value = [&](int n) -> uint4 {
                    Pair p[PAIRS];
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) p[i] = e[n * PAIRS + i] * gg;
                    return Gr::pack(p);
                };
                if (!taught) {      // whatever the logits hold
#pragma unroll
                    for (int i = 0; i < NG * PAIRS; ++i) e[i] = {0.0f, 0.0f};
                    edge = 0.0f;
                }
                if (a.segments == 1 && d->seg[0].aligned) {
                    char *to = reinterpret_cast<char *>(d->seg[0].out) + size_t(tid) * 16;
#pragma unroll
                    for (int n = 0; n < NG; ++n)
                        if (uint32_t(tid + n * kDistillConsumers) < groups && stores(0, to + n * kDistillConsumers * 16, 16))
                            st_stream_v4(to + n * kDistillConsumers * 16, value(n));
                } else {
#pragma unroll
                    for (int n = 0; n < NG; ++n) {
                        const uint32_t g16 = tid + n * kDistillConsumers;
                        if (g16 >= groups) continue;
                        uint32_t sg = 0;
                        while (sg + 1 < a.segments && d->seg[sg + 1].first <= g16) ++sg;
                        const uintptr_t to = uintptr_t(d->seg[sg].out) + uintptr_t(g16 - d->seg[sg].first) * 16;
                        if (!stores(sg, reinterpret_cast<const void *>(to), 16)) continue;
                        const uint4 v = value(n);
                        if (d->seg[sg].aligned) {
                            st_stream_v4(reinterpret_cast<void *>(to), v);
                        } else {
                            float f[VEC];
                            Tr::unpack(v, f);
#pragma unroll
                            for (int i = 0; i < VEC; ++i) Tr::store1(reinterpret_cast<void *>(to), i, f[i]);
                        }
                    }
                }
                if (a.edges && uint32_t(tid) < a.segments * 2 * VEC && d->edge_out[tid] &&
                    stores(tid / (2 * VEC), reinterpret_cast<const void *>(uintptr_t(d->edge_out[tid])), 16 / VEC))
                    Tr::store1(reinterpret_cast<void *>(uintptr_t(d->edge_out[tid])), 0, edge * gg.x);
            };
            float row_m = 0.0f, inv = 0.0f, factor = 0.0f;
            bool taught = true;
            if constexpr (FWD) {
                for (uint32_t c = 0; c < a.chunks; ++c) {
                    arrive();
                    if (!ok) break;
#pragma unroll
                    for (int part = 0; part < NG; part += TAKE) {
                        const float cm = Gr::value(take(part));
                        const float bm = fmaxf(m, part == 0 ? fmaxf(cm, edge) : cm), to = finite_max(bm);
                        sum *= ex2((m - to) * c2);            // nothing yet: 0 * 2^-inf
                        m = bm;
                        Pair acc = {0.0f, 0.0f}, acc2 = {0.0f, 0.0f};
                        if (part == 0) acc.x = edge = ex2((edge - to) * c2);
#pragma unroll
                        for (int i = 0; i < TAKE * PAIRS; i += 2) {
                            e[i] = ex2((e[i] + Pair{-to, -to}) * cc);
                            e[i + 1] = ex2((e[i + 1] + Pair{-to, -to}) * cc);
                            acc = acc + e[i];
                            acc2 = acc2 + e[i + 1];
                        }
                        acc = acc + acc2;
                        sum += acc.x + acc.y;
                    }
                }
                if (!ok) break;
                const float wm = warp_max(m);
                const float ws = warp_sum(sum * ex2((m - finite_max(wm)) * c2));
                // the loss alone does not wait for this row's sums, only for those of two rows back
                if (!BWD && k >= kDistillLag) {
                    if (!wait_sums(a, sh, k - kDistillLag, 11, item)) break;
                    if (warp == 0 && q == (k - kDistillLag) % a.pieces) finish_row((k - kDistillLag) % kDistillSlots, div_by(item - kDistillLag * stride, a.by_pieces));
                }
                const uint32_t to = k % kDistillSlots;
                if (lane < int(a.pieces))
                    send2(remote(smem_addr(&sh.sums[to].warp[q][warp]), lane), remote(smem_addr(&sh.sums_in[to]), lane), wm, ws);
                if constexpr (BWD) {
                    if (!wait_sums(a, sh, k, 12, item)) break;
                    const float total = total_of(to, row_m);
                    row_m = finite_max(row_m);
                    inv = total == 0.0f ? 0.0f : 1.0f / total;    // a row of nothing but -inf: p = 0
                    taught = sh.sums[to].teacher[q][0].w != 0.0f;
                    factor = sh.sums[to].teacher[q][1].y * a.temperature;
                }
            }
            if constexpr (BWD) {
                if (FWD && a.chunks == 1) {
                    put(inv * ex2((m - row_m) * c2) * factor, taught);
                } else {
                    for (uint32_t c = 0; c < a.chunks; ++c) {
                        arrive();
                        if (!ok) break;
                        take(0);
                        if (!FWD && c == 0) {
                            ok = __all_sync(0xffffffffu, distill_wait(a, sh, &sh.taught[slot], parity, 13, item));
                            if (!ok) break;
                            const float mx = sh.row_max[slot];
                            row_m = finite_max(mx);
                            inv = mx == -INFINITY ? 0.0f : expf(-sh.row_log_sum[slot]);
                            factor = sh.weight[slot] * a.temperature;
                            taught = sh.teacher_sum[slot] != 0.0f;
                        }
                        edge = ex2((edge - row_m) * c2);
#pragma unroll
                        for (int i = 0; i < NG * PAIRS; ++i) e[i] = ex2((e[i] + Pair{-row_m, -row_m}) * cc);
                        put(inv * factor, taught);
                    }
                    if (!ok) break;
                }
                if (tid == 0) {
                    sh.used_max[slot] = row_m;
                    sh.used_inv[slot] = inv;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.stored[slot]));
            }
        }
        if constexpr (!BWD) {
            // the last rows' losses
            for (uint32_t j = k > kDistillLag ? k - kDistillLag : 0u; j < k; ++j) {
                const uint32_t item = blockIdx.x + j * stride, row = div_by(item, a.by_pieces), q = item - row * a.pieces;
                if (!wait_sums(a, sh, j, 14, item)) break;
                if (warp == 0 && q == j % a.pieces) finish_row(j % kDistillSlots, row);
            }
        }
    }

    // A CTA that gave up: its copies in flight land before it goes, and what
    // the other CTAs of the row still send has a while to arrive.
    __syncthreads();
    if (warp == kDistillWarps && *static_cast<volatile int *>(&sh.dead)) {
        const uint64_t t0 = global_ns();
        for (uint32_t n = issued > S ? issued - S : 0; n < issued; ++n)
            while (!mbar_try_wait(smem_addr(&sh.full[n % S]), (n / S) & 1))
                if (global_ns() - t0 > uint64_t(a.wait_ns) + 1000000) break;
        while (FWD && global_ns() - t0 < 1000000) {
        }
    }
    if (FWD) {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}

// Shared-memory and cluster attributes, set once per device, and the clusters
// of each size that fit the GPU at once.
template <typename T, int PM, int PASS, int HELD>
static cudaError_t distill_residents(const Launch &L, const cudaLaunchConfig_t &cfg, uint32_t pieces, uint32_t stages, uint32_t *ctas)
{
    static std::atomic<unsigned long long> done{0};
    static std::atomic<int> fit[DistillShape<PASS>::cluster + 1][DistillShape<PASS>::stages + 1];
    static std::atomic<int> fit_device{-1};
    auto kern = distill_kernel<T, PM, PASS, HELD>;
    const unsigned long long bit = (L.device >= 0 && L.device < 64) ? (1ull << L.device) : 0ull;
    if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
        cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(DistillShape<PASS>::smem));
        if (err == cudaSuccess) err = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (err != cudaSuccess) return err;
        if (bit) done.fetch_or(bit, std::memory_order_acq_rel);
    }
    if (!(PASS & CCL_PASS_FORWARD)) {
        *ctas = DistillShape<PASS>::ctas * uint32_t(L.num_sms);
        return cudaSuccess;
    }
    int n = fit_device.load(std::memory_order_acquire) == L.device ? fit[pieces][stages].load(std::memory_order_acquire) : 0;
    if (n == 0) {
        const cudaError_t err = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        if (err != cudaSuccess) return err;
        if (n < 1) return cudaErrorInvalidConfiguration;
        int none = -1;
        if (fit_device.compare_exchange_strong(none, L.device, std::memory_order_acq_rel) || none == L.device)
            fit[pieces][stages].store(n, std::memory_order_release);
    }
    *ctas = uint32_t(n) * pieces;
    return cudaSuccess;
}

template <typename T, int PM, int PASS, int HELD>
static cudaError_t distill_held(const Launch &L, const DistillLaunch &N, LaunchInfo *info)
{
    DistillArgs<PM> a;
    fill_shards(&a.s, L, N.rows, N.vocab, N.ld, kSiteDistill);
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
    constexpr uint32_t VEC = Traits<T>::VEC;
    a.edges = a.s.q % VEC != 0 || a.s.rem != 0 || N.ld % VEC != 0;
    for (int r = 0; r < L.p; ++r) a.edges = a.edges || uintptr_t(L.src[r]) % 16 != 0;
    a.wait_ns = L.wait_limit_ns > 0 ? L.wait_limit_ns : 2000000000LL;
    a.stall_test = L.stall_test;
    const uint32_t p = a.s.p, groups = widest_groups<T>(a.s);
    // Pieces: few enough groups that a stage holds one, in a cluster of the
    // portable eight CTAs where that will do and of sixteen where not (a
    // gradient alone needs no cluster, so any number); then, with fewer CTAs
    // than two per SM, more and smaller pieces, for latency (8 x 32000 f32:
    // 3.9 us, else 4.2).
    // Several shards a piece where they fit a stage together and the rows keep
    // every SM at work, as an item's cost hardly depends on its size: 2048 x
    // 32000 bf16 on 8 ranks 70 us, 193 with a shard a piece; 160 rows 10.4,
    // 21.2; the loss alone 30, 108; the gradient alone 55, 116.
    using Shape = DistillShape<PASS>;
    a.segments = (p + Shape::cluster - 1) / Shape::cluster;
    for (uint32_t more = a.segments + 1; more <= Shape::segments && more * groups <= kDistillStage; ++more) {
        const uint32_t pieces = (p + more - 1) / more;
        if (N.rows * pieces >= 2 * uint64_t(L.num_sms) && pieces < (p + a.segments - 1) / a.segments) a.segments = more;
    }
    a.parts = 1;
    auto per_part = [&](uint32_t parts) { return (groups + parts - 1) / parts; };
    uint32_t cap = kDistillStage / a.segments;
    if (a.segments == 1) {
        const uint32_t most = (PASS & CCL_PASS_FORWARD) ? Shape::cluster / p : (1u << 20) / p, portable = (PASS & CCL_PASS_FORWARD) ? 8 / p : most;
        while (a.parts < most && per_part(a.parts) > cap) ++a.parts;
        while (a.parts < portable && N.rows * p * a.parts < 2 * uint64_t(L.num_sms) && per_part(a.parts) > kDistillConsumers) ++a.parts;
    }
    a.pieces = a.segments == 1 ? p * a.parts : (p + a.segments - 1) / a.segments;
    a.chunks = (per_part(a.parts) + cap - 1) / cap;
    if (a.chunks < 1) a.chunks = 1;
    a.span = 0;
    a.groups = groups;
    // The loss alone: fewer pieces that go over the shards' bounds (2048 x
    // 80768 bf16 on 8 ranks, 8 entries, five for eight: 69 us, 109; with the
    // gradient, whose stores then have to look for their shard, 212 and 180).
    const uint64_t total = uint64_t(groups) * p;
    for (uint64_t pieces = (total + kDistillStage - 1) / kDistillStage; Shape::loss_alone && groups && pieces < a.pieces; ++pieces) {
        if (pieces > Shape::cluster || N.rows * pieces < 2 * uint64_t(L.num_sms)) continue;
        const uint64_t span = (total + pieces - 1) / pieces;
        uint64_t most = 1;      // shards that a piece touches
        for (uint64_t at = 0; at < total; at += span) {
            const uint64_t end = at + span < total ? at + span : total, touched = (end - 1) / groups - at / groups + 1;
            if (touched > most) most = touched;
        }
        if (most < 2 || most > Shape::segments) continue;
        a.segments = uint32_t(most);
        a.parts = a.chunks = 1;
        a.pieces = uint32_t(pieces);
        a.span = uint32_t(span);
        break;
    }
    if (N.rows * a.pieces > 0x7fffffffull) return kTooManyPieces;
    a.items = uint32_t(N.rows * a.pieces);
    a.by_pieces = fast_div(a.pieces);
    a.by_parts = fast_div(a.parts);
    a.by_segments = fast_div(a.segments);
    a.by_groups = fast_div(groups ? groups : 1);
    a.share = (a.k + a.pieces - 1) / a.pieces;
    const uint32_t in_registers = 32 * HELD, share = Shape::loss_alone ? a.share : a.k;
    const size_t entries = size_t(a.kpad) * ((Shape::loss_alone ? 0 : 24) + (share > in_registers ? 12 * kDistillTeachers<HELD> : 0));
    a.stages = Shape::stages;
    while (a.stages > 1 && a.stages * size_t(kDistillStageBytes) + entries + sizeof(DistillShared<PASS>) + 1024 > Shape::smem) --a.stages;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kDistillThreads<HELD>);
    cfg.dynamicSmemBytes = a.stages * size_t(kDistillStageBytes) + entries;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.pieces;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (PASS & CCL_PASS_FORWARD) ? 2 : 1;
    cfg.gridDim = dim3(a.pieces);
    uint32_t ctas = 0;
    cudaError_t err = distill_residents<T, PM, PASS, HELD>(L, cfg, a.pieces, a.stages, &ctas);
    if (err != cudaSuccess) return err;
    cfg.gridDim = dim3(a.items < ctas ? a.items : ctas);
    err = cudaLaunchKernelEx(&cfg, distill_kernel<T, PM, PASS, HELD>, a);
    if (err != cudaSuccess) return err;
    info->kernel = "distill_topk";
    info->grid = int(cfg.gridDim.x);
    info->block = kDistillThreads<HELD>;
    info->smem = cfg.dynamicSmemBytes;
    info->kernels = 1;
    return cudaGetLastError();
}

template <typename T, int PM, int PASS>
static cudaError_t distill_shape(const Launch &L, const DistillLaunch &N, LaunchInfo *info)
{
    // (the loss alone: each piece has a share of the entries)
    if constexpr (PASS != CCL_PASS_FORWARD) {
        if (N.k > 128) return distill_held<T, PM, PASS, 3>(L, N, info);
        if (N.k > 64) return distill_held<T, PM, PASS, 4>(L, N, info);
    }
    return distill_held<T, PM, PASS, 2>(L, N, info);
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
    return L.p <= 8 ? distill_pass<T, 8>(L, N, info) : distill_pass<T, kMaxRanks>(L, N, info);
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
