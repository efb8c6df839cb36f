// Tokens to the rows of their experts and back: dispatch, combine and
// combine's gradient over p ranks' buffers.
//
//   dispatch  row[slot_tj] = w_tj x_t
//   combine   y_t          = sum_j w_tj row[slot_tj]
//   gradient  drow[slot_tj] = w_tj dy_t,  dw_tj = <dy_t, row[slot_tj]>
// Each is driven by the tokens: a team of 8 to 256 threads takes one, so a
// token's row is read (or written) once and its k expert rows once each, which
// is all the traffic there has to be.  A thread loads a batch of KB choices of
// UN units before it uses the first.
#include "logits.cuh"

namespace ccl {

constexpr unsigned kSiteExperts = 11;
constexpr int kRowsThreads = 256;
constexpr int kRowsTeam = 8;       // threads of a team, at least

template <int PM>
struct RowsArgs {
    const void *in[PM];
    void *out[PM];
    const int32_t *slots[PM];
    const float *weights[PM];
    const void *experts[PM];
    float *dweights[PM];
    uint64_t hidden;
    uint32_t rows, p, k, capacity, slot_end;   // slot_end: p * capacity
    FastDiv by_rows, by_capacity;
    int weighted;
    int team_shift;       // a team has 2^team_shift threads
    // checked build:
    unsigned *status;
    uint32_t held;        // tokens that every token buffer and list has: `rows`, or one less where the debug hook wants the checks to fail
};

template <int PM>
__device__ __forceinline__ bool token_held(const RowsArgs<PM> &a, const void *buf, const void *at, uint32_t bytes, uint32_t element)
{
    return !kBoundsCheck || in_buffer(at, bytes, buf, uint64_t(a.held) * a.hidden * element, a.status, kSiteExperts);
}
template <int PM>
__device__ __forceinline__ bool row_of_expert_held(const RowsArgs<PM> &a, const void *buf, const void *at, uint32_t bytes, uint32_t element)
{
    return !kBoundsCheck || in_buffer(at, bytes, buf, uint64_t(a.capacity) * a.hidden * element, a.status, kSiteExperts);
}
template <int PM>
__device__ __forceinline__ bool entry_held(const RowsArgs<PM> &a, uint64_t entry)
{
    return in_bounds(entry < uint64_t(a.held) * a.k, a.status, kSiteExperts, entry);
}

// A row anywhere in memory, in 16-byte groups that lie on 16-byte boundaries:
// group g has columns g VEC - shift and on.
template <typename T>
struct RowView {
    static constexpr int VEC = Traits<T>::VEC, S = 16 / VEC;
    char *base;            // the boundary at or below the row's begin
    int shift;             // elements between the boundary and the row
    __device__ __forceinline__ explicit RowView(const void *row)
    {
        base = reinterpret_cast<char *>(uintptr_t(row) & ~uintptr_t(15));
        shift = int(uintptr_t(row) & 15) / S;
    }
    __device__ __forceinline__ char *at(int g) const { return base + int64_t(g) * 16; }
    __device__ __forceinline__ char *column(int c) const { return base + int64_t(shift + c) * S; }
    // The columns of group g of a row with shift `other`: two groups (a neighbouring thread has one of them too) and a shift
    // that is the same for all of the two rows.  For groups in `inner` both lie in the row.
    __device__ __forceinline__ uint4 load_for(int g, int other) const
    {
        int by = (shift - other) * S;
        if (by < 0) {
            by += 16;
            --g;
        }
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(at(g)));
        if (by == 0) return a;
        const uint4 b = __ldg(reinterpret_cast<const uint4 *>(at(g + 1)));
        uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (by & 8)
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        if (by & 4)
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        if (by & 2)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// The groups of a written row of `width` columns that are moved whole, [2,
// last): two groups from its begin and one before its last whole one, whatever
// the shift of the row that is read, the groups read lie in that row.  The
// columns before and after them, 16 at most each, go element by element, a thread each; so do all
// columns of rows without such groups.
template <typename T>
struct Inner {
    static constexpr int VEC = Traits<T>::VEC;
    int last, head, tail, edges;     // columns [0, head) and from `tail` on are the edges
    __device__ __forceinline__ Inner(int shift, int width)
    {
        last = (shift + width) / VEC - 1;
        head = 2 * VEC - shift;
        tail = last * VEC - shift;
        if (last <= 2) head = tail = width;
        edges = head + width - tail;
    }
    __device__ __forceinline__ int edge(int n) const { return n < head ? n : tail + n - head; }
};

// One choice of a team's token: where its row begins, and its weight.
struct Choice {
    char *row;            // null: none
    float weight;
    uint32_t rank;
};

// A team of threads, its token and its choices.
template <int PM>
struct Team {
    uint32_t thread, threads;   // of the team
    uint32_t rank, token;
    uint64_t first, end;        // the team's units: of a row, or of a row and as many more as it may lie over
    bool on;                    // it has a token
    Choice *list;

    // The sums of a team's threads, N of them: its lanes' in every thread of a warp, or of the team where that is less ...
    template <int N>
    __device__ __forceinline__ void lanes(float (&v)[N]) const
    {
        if (threads >= 32) {
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
        } else {
            for (uint32_t o = threads / 2; o > 0; o >>= 1)
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
        }
    }
    // ... left in parts[part()] by its first, and added up from parts[first_part()] on.
    __device__ __forceinline__ uint32_t part() const { return threadIdx.x / min(threads, 32u); }
    __device__ __forceinline__ bool leads() const { return thread % 32 == 0; }
    __device__ __forceinline__ uint32_t parts() const { return max(1u, threads / 32); }
    __device__ __forceinline__ uint32_t first_part() const { return (threadIdx.x - thread) / min(threads, 32u); }

    // `of` has the experts' buffers; `list` room for the choices of all teams.
    __device__ __forceinline__ Team(const RowsArgs<PM> &a, const void *const *of, uint32_t S, uint64_t units, Choice *all)
    {
        threads = 1u << a.team_shift;
        thread = threadIdx.x & (threads - 1);
        const uint32_t team = threadIdx.x >> a.team_shift, t = blockIdx.x * (kRowsThreads >> a.team_shift) + team;
        on = t < a.rows * a.p;
        rank = on ? div_by(t, a.by_rows) : 0;
        token = t - rank * a.rows;
        first = units * blockIdx.y / gridDim.y + thread;
        end = on ? units * (blockIdx.y + 1) / gridDim.y : 0;
        list = all + team * a.k;
        for (uint32_t j = thread; j < a.k; j += threads) {
            const uint64_t entry = uint64_t(token) * a.k + j;
            Choice c = {nullptr, 1.0f, 0};
            if (on && entry_held(a, entry)) {
                const uint32_t slot = uint32_t(a.slots[rank][entry]);
                if (a.weighted) c.weight = a.weights[rank][entry];
                if (slot < a.slot_end) {
                    c.rank = div_by(slot, a.by_capacity);
                    c.row = static_cast<char *>(const_cast<void *>(of[c.rank])) + uint64_t(slot - c.rank * a.capacity) * a.hidden * S;
                }
            }
            list[j] = c;
        }
        __syncthreads();
    }
};

template <typename T, int PM, int UN>
__global__ void __launch_bounds__(kRowsThreads) dispatch_kernel(const __grid_constant__ RowsArgs<PM> a)
{
    using Tr = Traits<T>;
    constexpr uint32_t VEC = Tr::VEC, S = 16 / VEC;
    extern __shared__ Choice lists[];
    grid_dependency_wait();
    grid_dependents_launch();
    const Team<PM> t(a, a.out, S, a.hidden / VEC, lists);
    const char *token = static_cast<const char *>(a.in[t.rank]) + uint64_t(t.token) * a.hidden * S;
    for (uint64_t u = t.first; u < t.end; u += UN * t.threads) {
        uint4 v[UN];
#pragma unroll
        for (int n = 0; n < UN; ++n) {
            const char *at = token + (u + n * t.threads) * 16;
            if (u + n * t.threads < t.end && token_held(a, a.in[t.rank], at, 16, S)) v[n] = ld_stream_v4(at);
        }
        for (uint32_t j = 0; j < a.k; ++j) {
            const Choice c = t.list[j];
            if (!c.row) continue;
#pragma unroll
            for (int n = 0; n < UN; ++n) {
                const uint64_t at = (u + n * t.threads) * 16;
                if (u + n * t.threads >= t.end || !token_held(a, a.in[t.rank], token + at, 16, S) ||
                    !row_of_expert_held(a, a.out[c.rank], c.row + at, 16, S))
                    continue;
                uint4 w = v[n];
                if constexpr (!std::is_same<T, I32>::value) {
                    if (a.weighted) {
                        float f[int(VEC)];
                        Tr::unpack(w, f);
#pragma unroll
                        for (int i = 0; i < int(VEC); ++i) f[i] = __fmul_rn(f[i], c.weight);
                        w = Tr::pack(f);
                    }
                }
                st_stream_v4(c.row + at, w);
            }
        }
    }
}

template <typename T, int PM, int KB, int UN>
__global__ void __launch_bounds__(kRowsThreads, KB * UN == 8 ? 3 : 4) combine_kernel(const __grid_constant__ RowsArgs<PM> a)
{
    using Tr = Traits<T>;
    constexpr uint32_t VEC = Tr::VEC, S = 16 / VEC;
    extern __shared__ Choice lists[];
    grid_dependency_wait();
    grid_dependents_launch();
    const Team<PM> t(a, a.in, S, a.hidden / VEC, lists);
    char *token = static_cast<char *>(a.out[t.rank]) + uint64_t(t.token) * a.hidden * S;
    for (uint64_t u = t.first; u < t.end; u += UN * t.threads) {
        float sum[UN][int(VEC)];
#pragma unroll
        for (int n = 0; n < UN; ++n)
#pragma unroll
            for (int i = 0; i < int(VEC); ++i) sum[n][i] = 0.0f;
        for (uint32_t first = 0; first < a.k; first += KB) {
            uint4 z[KB][UN];
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const Choice c = first + j < a.k ? t.list[first + j] : Choice{nullptr, 0.0f, 0};
#pragma unroll
                for (int n = 0; n < UN; ++n) {
                    const char *at = c.row + (u + n * t.threads) * 16;
                    z[j][n] = make_uint4(0, 0, 0, 0);
                    if (c.row && u + n * t.threads < t.end && row_of_expert_held(a, a.in[c.rank], at, 16, S)) z[j][n] = ld_stream_v4(at);
                }
            }
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                if (first + j >= a.k) break;
                const Choice c = t.list[first + j];
                if (!c.row) continue;
#pragma unroll
                for (int n = 0; n < UN; ++n) {
                    float f[int(VEC)];
                    Tr::unpack(z[j][n], f);
#pragma unroll
                    for (int i = 0; i < int(VEC); ++i) sum[n][i] = fmaf(c.weight, f[i], sum[n][i]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < UN; ++n) {
            char *at = token + (u + n * t.threads) * 16;
            if (u + n * t.threads < t.end && token_held(a, a.out[t.rank], at, 16, S)) st_stream_v4(at, Tr::pack(sum[n]));
        }
    }
}

template <typename T, int PM, int KB, int UN>
__global__ void __launch_bounds__(kRowsThreads, KB * UN == 8 ? 3 : 4) combine_grad_kernel(const __grid_constant__ RowsArgs<PM> a)
{
    using Tr = Traits<T>;
    constexpr uint32_t VEC = Tr::VEC, S = 16 / VEC;
    extern __shared__ Choice lists[];
    __shared__ float parts[kRowsThreads / kRowsTeam][KB];
    grid_dependency_wait();
    grid_dependents_launch();
    const Team<PM> t(a, a.out, S, a.hidden / VEC, lists);
    const char *token = static_cast<const char *>(a.in[t.rank]) + uint64_t(t.token) * a.hidden * S;
    for (uint32_t first = 0; first < a.k; first += KB) {
        float sum[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) sum[j] = 0.0f;
        for (uint64_t u = t.first; u < t.end; u += UN * t.threads) {
            uint4 v[UN], z[KB][UN];
#pragma unroll
            for (int n = 0; n < UN; ++n) {
                const char *at = token + (u + n * t.threads) * 16;
                v[n] = make_uint4(0, 0, 0, 0);
                if (u + n * t.threads < t.end && token_held(a, a.in[t.rank], at, 16, S)) v[n] = ld_stream_v4(at);
            }
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const Choice c = first + j < a.k ? t.list[first + j] : Choice{nullptr, 0.0f, 0};
                const char *row = c.row ? static_cast<const char *>(a.experts[c.rank]) + (c.row - static_cast<char *>(a.out[c.rank])) : nullptr;
#pragma unroll
                for (int n = 0; n < UN; ++n) {
                    const char *at = row + (u + n * t.threads) * 16;
                    z[j][n] = make_uint4(0, 0, 0, 0);
                    if (c.row && u + n * t.threads < t.end && row_of_expert_held(a, a.experts[c.rank], at, 16, S)) z[j][n] = ld_stream_v4(at);
                }
            }
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                if (first + j >= a.k) break;
                const Choice c = t.list[first + j];
                if (!c.row) continue;
#pragma unroll
                for (int n = 0; n < UN; ++n) {
                    char *at = c.row + (u + n * t.threads) * 16;
                    float f[int(VEC)], g[int(VEC)];
                    Tr::unpack(v[n], f);
                    Tr::unpack(z[j][n], g);
#pragma unroll
                    for (int i = 0; i < int(VEC); ++i) sum[j] = fmaf(f[i], g[i], sum[j]);
#pragma unroll
                    for (int i = 0; i < int(VEC); ++i) f[i] = __fmul_rn(f[i], c.weight);
                    if (u + n * t.threads < t.end && token_held(a, a.in[t.rank], token + (u + n * t.threads) * 16, 16, S) &&
                        row_of_expert_held(a, a.out[c.rank], at, 16, S))
                        st_stream_v4(at, Tr::pack(f));
                }
            }
        }
        // the team's sums: its warps', in order
        t.lanes(sum);
        if (t.leads())
#pragma unroll
            for (int j = 0; j < KB; ++j) parts[t.part()][j] = sum[j];
        __syncthreads();
        if (t.on && t.thread < KB && first + t.thread < a.k) {
            float s = 0.0f;
            for (uint32_t w = 0; w < t.parts(); ++w) s += parts[t.first_part() + w][t.thread];
            const uint64_t entry = uint64_t(t.token) * a.k + first + t.thread;
            if (entry_held(a, entry)) a.dweights[t.rank][entry] = t.list[first + t.thread].row ? s : 0.0f;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Rows that are no 16-byte groups, or do not begin on a boundary.  A load at
// any column is two aligned ones and a shift; what is written goes by the
// groups of the row that is written.  Measured (us; against accesses of one
// element, or of 4 bytes where they are aligned): combine, 2 x 4000 x 1001 bf16, k=4, 36 -> 23.5; its gradient
// 94 -> 39, of 3 x 12400 x 731 bf16, k=2, 224 -> 95; dispatch, 3 x 1111 x 1001 f32, 7.6 -> 7.5.  With choices sorted by expert
// 2 x 4000 x 1001 bf16, k=4, takes 13.7 (dispatch, copy rate 11.7), 17.0 (combine, 11.8) and 34 (gradient, 21.1).
// ---------------------------------------------------------------------------

// The checked build tests rows as a whole here: the views keep to them.
template <typename T, int PM>
__device__ __forceinline__ bool rows_held(const RowsArgs<PM> &a, uint32_t rank, uint32_t token, const void *tokens, const Choice &c, const void *expert, const void *row)
{
    constexpr uint32_t S = 16 / Traits<T>::VEC;
    const uint64_t bytes = a.hidden * S;
    if (!kBoundsCheck) return true;
    return in_buffer(static_cast<const char *>(tokens) + token * bytes, bytes, tokens, a.held * bytes, a.status, kSiteExperts) &&
           (!c.row || in_buffer(row, bytes, expert, a.capacity * bytes, a.status, kSiteExperts));
}

template <typename T, int PM, bool GRAD>
__global__ void __launch_bounds__(kRowsThreads, 5) scatter_odd_kernel(const __grid_constant__ RowsArgs<PM> a)
{
    using Tr = Traits<T>;
    constexpr int VEC = Tr::VEC, S = 16 / VEC, KB = 8;
    constexpr bool RAW = std::is_same<T, I32>::value;
    extern __shared__ Choice lists[];
    __shared__ float parts[kRowsThreads / kRowsTeam][KB];
    grid_dependency_wait();
    grid_dependents_launch();
    const Team<PM> t(a, a.out, S, a.hidden / VEC + 2, lists);
    const int width = int(a.hidden), thread = int(t.thread), threads = int(t.threads);
    const char *token = static_cast<const char *>(a.in[t.rank]) + uint64_t(t.token) * a.hidden * S;
    const RowView<T> x(token);
    for (uint32_t first = 0; first < a.k; first += KB) {
        for (uint32_t j = 0; j < KB && first + j < a.k; ++j) {
            const Choice c = t.list[first + j];
            float sum = 0.0f;
            const char *row = c.row && GRAD ? static_cast<const char *>(a.experts[c.rank]) + (c.row - static_cast<char *>(a.out[c.rank])) : nullptr;
            if (c.row && t.on && rows_held<T>(a, t.rank, t.token, a.in[t.rank], c, a.out[c.rank], c.row) &&
                (!GRAD || rows_held<T>(a, t.rank, t.token, a.in[t.rank], c, a.experts[c.rank], row))) {
                const RowView<T> to(c.row), z(row);
                const Inner<T> in(to.shift, width);
                for (int g = 2 + int(t.first); g < in.last && g - 2 < int(t.end); g += threads) {
                    uint4 v = x.load_for(g, to.shift);
                    if constexpr (!RAW) {
                        if (GRAD || a.weighted) {
                            float f[VEC];
                            if constexpr (GRAD) {
                                const uint4 h = z.shift == to.shift ? ld_stream_v4(z.at(g)) : z.load_for(g, to.shift);
                                float e[VEC];
                                Tr::unpack(h, e);
                                Tr::unpack(v, f);
#pragma unroll
                                for (int i = 0; i < VEC; ++i) sum = fmaf(f[i], e[i], sum);
                            } else {
                                Tr::unpack(v, f);
                            }
#pragma unroll
                            for (int i = 0; i < VEC; ++i) f[i] = __fmul_rn(f[i], c.weight);
                            if (a.weighted) v = Tr::pack(f);
                        }
                    }
                    st_stream_v4(to.at(g), v);
                }
                if (blockIdx.y == 0)
                    for (int n = thread; n < in.edges; n += threads) {
                        const int col = in.edge(n);
                        if constexpr (RAW) {
                            *reinterpret_cast<uint32_t *>(to.column(col)) = *reinterpret_cast<const uint32_t *>(x.column(col));
                        } else if (!GRAD && !a.weighted) {
                            using Bits = typename std::conditional<S == 2, uint16_t, uint32_t>::type;
                            *reinterpret_cast<Bits *>(to.column(col)) = *reinterpret_cast<const Bits *>(x.column(col));
                        } else {
                            const float f = Tr::load1(x.column(col), 0);
                            if constexpr (GRAD) sum = fmaf(f, Tr::load1(z.column(col), 0), sum);
                            Tr::store1(to.column(col), 0, __fmul_rn(f, c.weight));
                        }
                    }
            }
            if constexpr (GRAD) {
                float one[1] = {sum};
                t.lanes(one);
                if (t.leads()) parts[t.part()][j] = one[0];
            }
        }
        if constexpr (GRAD) {
            __syncthreads();
            if (t.on && t.thread < KB && first + t.thread < a.k) {
                float s = 0.0f;
                for (uint32_t w = 0; w < t.parts(); ++w) s += parts[t.first_part() + w][t.thread];
                const uint64_t entry = uint64_t(t.token) * a.k + first + t.thread;
                if (entry_held(a, entry)) a.dweights[t.rank][entry] = s;
            }
            __syncthreads();
        }
    }
}

template <typename T, int PM>
__global__ void __launch_bounds__(kRowsThreads, 5) combine_odd_kernel(const __grid_constant__ RowsArgs<PM> a)
{
    using Tr = Traits<T>;
    constexpr int VEC = Tr::VEC, S = 16 / VEC, KB = 2;
    extern __shared__ Choice lists[];
    grid_dependency_wait();
    grid_dependents_launch();
    const Team<PM> t(a, a.in, S, a.hidden / VEC + 2, lists);
    if (!t.on) return;
    const int width = int(a.hidden), thread = int(t.thread), threads = int(t.threads);
    const RowView<T> to(static_cast<char *>(a.out[t.rank]) + uint64_t(t.token) * a.hidden * S);
    if (!rows_held<T>(a, t.rank, t.token, a.out[t.rank], Choice{nullptr, 0.0f, 0}, nullptr, nullptr)) return;
    const Inner<T> in(to.shift, width);
    auto held = [&](const Choice &c) { return c.row && rows_held<T>(a, t.rank, t.token, a.out[t.rank], c, a.in[c.rank], c.row); };
    for (int g = 2 + int(t.first); g < in.last && g - 2 < int(t.end); g += threads) {
        float sum[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
        for (uint32_t first = 0; first < a.k; first += KB) {
            uint4 z[KB];
            float weight[KB];
            bool has[KB];
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const Choice c = first + j < a.k ? t.list[first + j] : Choice{nullptr, 0.0f, 0};
                has[j] = held(c);
                weight[j] = c.weight;
                if (has[j]) z[j] = RowView<T>(c.row).load_for(g, to.shift);
            }
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                if (!has[j]) continue;
                float f[VEC];
                Tr::unpack(z[j], f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum[i] = fmaf(weight[j], f[i], sum[i]);
            }
        }
        st_stream_v4(to.at(g), Tr::pack(sum));
    }
    if (blockIdx.y == 0)
        for (int n = thread; n < in.edges; n += threads) {
            const int col = in.edge(n);
            float sum = 0.0f;
#pragma unroll 4
            for (uint32_t j = 0; j < a.k; ++j) {
                const Choice c = t.list[j];
                if (held(c)) sum = fmaf(c.weight, Tr::load1(c.row, col), sum);
            }
            Tr::store1(to.column(col), 0, sum);
        }
}

// KB, UN: batches of the aligned kernels; KB 0: the others.
template <typename T, int PM, int KB, int UN>
static cudaError_t rows_launch(const Launch &L, const RowsLaunch &N, LaunchInfo *info)
{
    RowsArgs<PM> a = {};
    for (int r = 0; r < L.p; ++r) {
        a.in[r] = L.src[r];
        a.out[r] = L.dst[r];
        a.slots[r] = N.slots[r];
        a.weights[r] = N.weights ? N.weights[r] : nullptr;
        a.experts[r] = N.experts ? N.experts[r] : nullptr;
        a.dweights[r] = N.dweights ? N.dweights[r] : nullptr;
    }
    a.hidden = N.hidden;
    a.rows = uint32_t(N.rows);
    a.p = uint32_t(L.p);
    a.k = N.k;
    a.capacity = N.capacity;
    a.slot_end = N.capacity * uint32_t(L.p);
    a.by_rows = fast_div(a.rows);
    a.by_capacity = fast_div(N.capacity ? N.capacity : 1);
    a.weighted = N.weights ? 1 : 0;
    a.status = L.status;
    a.held = a.rows - (L.stall_test == 2 ? 1 : 0);
    // A team has four batches of units a thread (of odd rows two units), at least a warp where the row has a unit for each lane, and
    // more threads where there are few tokens or many choices.  (Rows of 8 units, 100000 bf16 tokens, k=2, with teams of 32 and 8:
    // dispatch 39, 12.4 us; combine 43, 13.5; its gradient 62, 20.)
    constexpr uint64_t VEC = Traits<T>::VEC;
    const uint64_t units = N.hidden / VEC + (KB ? 0 : 2), tokens = N.rows * uint64_t(L.p), sms = uint64_t(L.num_sms);
    a.team_shift = 3;
    while (a.team_shift < 8 && ((a.team_shift < 5 && (uint64_t(1) << a.team_shift) < units) || (uint64_t(KB ? 4 * UN : 2) << a.team_shift) < units ||
                                tokens >> (8 - a.team_shift) < 4 * sms || N.k > 32))
        ++a.team_shift;
    const uint32_t teams = kRowsThreads >> a.team_shift;
    const unsigned grid = unsigned((tokens + teams - 1) / teams);
    // few tokens: a row over several CTAs (the gradient's sums stay in one)
    uint64_t split = 1;
    if (N.op != ROWS_GRAD && grid < 4 * sms) {
        const uint64_t most = (units + kRowsThreads - 1) / kRowsThreads;
        split = (4 * sms + grid - 1) / grid;
        if (split > most) split = most;
        if (split < 1) split = 1;
    }
    const size_t smem = teams * N.k * sizeof(Choice);
    static std::atomic<unsigned long long> ready[3];
    void (*kern)(RowsArgs<PM>) = nullptr;
    if constexpr (std::is_same<T, I32>::value) {
        if constexpr (KB == 0) kern = scatter_odd_kernel<T, PM, false>;
        else kern = dispatch_kernel<T, PM, 4>;
    } else if constexpr (KB == 0) {
        kern = N.op == ROWS_DISPATCH ? scatter_odd_kernel<T, PM, false> : N.op == ROWS_COMBINE ? combine_odd_kernel<T, PM> : scatter_odd_kernel<T, PM, true>;
    } else {
        kern = N.op == ROWS_DISPATCH ? dispatch_kernel<T, PM, 4> : N.op == ROWS_COMBINE ? combine_kernel<T, PM, KB, UN> : combine_grad_kernel<T, PM, KB, UN>;
    }
    // (a kernel has 48 KB without asking, its own arrays among them: the gradient's are 1 KB)
    cudaError_t err = smem > 32 * 1024 ? allow_dynamic_smem(kern, 4096 * sizeof(Choice), L.device, ready[N.op]) : cudaSuccess;
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, unsigned(split));
    cfg.blockDim = dim3(kRowsThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kern, a);
    if (err != cudaSuccess) return err;
    info->kernel = N.op == ROWS_DISPATCH ? "expert_dispatch" : N.op == ROWS_COMBINE ? "expert_combine" : "expert_combine_grad";
    info->grid = int(grid * split);
    info->block = kRowsThreads;
    info->smem = smem;
    info->kernels = 1;
    return cudaSuccess;
}

// Batches by the number of choices.  Measured (graph replay, us; batches as
// choices x units):
//   combine, 8 x 4000 x 4096 bf16, k=2       2x4 102   2x2 106
//   combine's gradient, the same             2x4 160   2x2 162-170
//   gradient, 4 x 20000 x 512 f16, k=1       2x4 64    2x2 48: a row of 64 units fills two for each of 32 threads
//   gradient, 8 x 4000 x 2048 bf16, k=4      4x2 155
// with the registers held to three CTAs an SM for 8 units (four: 8 x 2048 x
// 7168 bf16, k=8, 602 and not 587) and to four for the others.
template <typename T, int PM>
static cudaError_t rows_batches(const Launch &L, const RowsLaunch &N, LaunchInfo *info)
{
    if (!L.vec) return rows_launch<T, PM, 0, 1>(L, N, info);
    if (PM > 8 || N.k > 4 || N.op == ROWS_DISPATCH) return rows_launch<T, PM, 8, 1>(L, N, info);
    if constexpr (PM <= 8) {
        if (N.k > 2) return rows_launch<T, PM, 4, 2>(L, N, info);
        return N.hidden < 128 * Traits<T>::VEC ? rows_launch<T, PM, 2, 2>(L, N, info) : rows_launch<T, PM, 2, 4>(L, N, info);
    }
    return cudaErrorInvalidValue;
}

template <typename T>
static cudaError_t rows_dtype(const Launch &L, const RowsLaunch &N, LaunchInfo *info)
{
    return L.p <= 8 ? rows_batches<T, 8>(L, N, info) : rows_batches<T, kMaxRanks>(L, N, info);
}

cudaError_t launch_expert_rows(const Launch &L, const RowsLaunch &N, LaunchInfo *info)
{
    switch (L.dtype) {
    case DT_F32: return rows_dtype<F32>(L, N, info);
    case DT_F16: return rows_dtype<F16>(L, N, info);
    case DT_BF16: return rows_dtype<BF16>(L, N, info);
    default: return rows_dtype<I32>(L, N, info);
    }
}

}  // namespace ccl
