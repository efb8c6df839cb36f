// Rank buffers that hold the shards of [rows, vocab] logits: rank r has the
// columns of balanced chunk r (the library's chunks: the larger ones first),
// row-major with a row stride of its own.
//
// A shard's row is worked through in 16-byte groups that lie on 16-byte
// boundaries of memory wherever the row itself begins: the groups that lie
// wholly inside the row are moved with 128-bit accesses, the elements before
// the first and after the last of them (fewer than a group each, the "edge")
// one by one, each by a thread of its own.  So odd vocabularies, odd strides
// and unaligned shards run at the speed of aligned ones.  A CTA (or a team of
// its warps) works on one shard, so addresses are uniform and the inner loops
// hold no arithmetic on ranks.
#pragma once

#include "device.cuh"

namespace ccl {

// Sites of the checked build's record (after BoundsSite).
constexpr unsigned kSiteRules = 8, kSiteDistill = 9, kSiteBalance = 10;

// in_bounds for an access to [at, at + bytes) of the buffer of `size` bytes that begins at `buf`.
__device__ __forceinline__ bool in_buffer(const void *at, uint64_t bytes, const void *buf, uint64_t size, unsigned *status, unsigned site)
{
    if constexpr (!kBoundsCheck) return true;
    const uint64_t from = uintptr_t(at) - uintptr_t(buf);       // (huge in front of it)
    return in_bounds(from <= size && bytes <= size - from, status, site, from);
}

// n / d for n < 2^31 by a multiplication.
struct FastDiv {
    uint32_t d, mul, shift;
};

inline FastDiv fast_div(uint32_t d)
{
    // shift = ceil(log2 d), mul = floor(2^32 (2^shift - d) / d) + 1: then
    // (mulhi(n, mul) + n) >> shift is the quotient (the round-up method of
    // Granlund and Montgomery, "Division by invariant integers using
    // multiplication")
    FastDiv f;
    f.d = d;
    f.shift = 0;
    while ((uint64_t(1) << f.shift) < d) ++f.shift;
    f.mul = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << f.shift) - d)) / d + 1);
    return f;
}

__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv &f)
{
    return (__umulhi(n, f.mul) + n) >> f.shift;
}

template <int PM>
struct Shards {
    const void *in[PM];
    void *out[PM];
    uint64_t ld;        // row stride in elements; 0: each shard is contiguous (its own width)
    uint64_t rows;
    uint32_t p, vocab;
    uint32_t q, rem;    // widths: q + 1 for the first rem ranks, then q
    FastDiv by_q1, by_q;
    // checked build:
    unsigned *status;   // the communicator's status block
    unsigned site;
    uint64_t held;      // rows that every buffer and list has: `rows`, or one less where the debug hook wants the checks to fail
};

template <int PM>
__device__ __forceinline__ uint32_t shard_width(const Shards<PM> &a, uint32_t r) { return a.q + (r < a.rem ? 1u : 0u); }
template <int PM>
__device__ __forceinline__ uint32_t shard_begin(const Shards<PM> &a, uint32_t r) { return r * a.q + min(r, a.rem); }

template <int PM>
__device__ __forceinline__ uint32_t rank_of_token(const Shards<PM> &a, uint32_t v)
{
    const uint32_t big = a.rem * (a.q + 1);
    return v < big ? div_by(v, a.by_q1) : a.rem + div_by(v - big, a.by_q);
}

// Bytes of rank r's buffers (checked build).
template <int PM>
__device__ __forceinline__ uint64_t shard_bytes(const Shards<PM> &a, uint32_t r, uint32_t element)
{
    const uint64_t w = shard_width(a, r);
    return a.held && w ? ((a.held - 1) * (a.ld ? a.ld : w) + w) * element : 0;
}

// Row `row` of a list with one entry, or one line of entries, a row.
template <int PM>
__device__ __forceinline__ bool row_held(const Shards<PM> &a, uint64_t row) { return in_bounds(row < a.held, a.status, a.site, row); }

// One row of one shard: of rank r's input or output buffer `buf`.
template <typename T, int PM>
struct ShardRow {
    static constexpr uint32_t VEC = Traits<T>::VEC, S = 16 / VEC;
    uintptr_t base;      // the 16-byte boundary at or below the row's first element
    uint32_t shift;      // elements between the boundary and the row
    uint32_t width;      // columns
    uint32_t first, end; // its whole groups are [first, end)
    const Shards<PM> &s; // (these for the checks)
    const void *buf;
    uint32_t rank;

    __device__ __forceinline__ ShardRow(const Shards<PM> &a, const void *of, uint32_t r, uint64_t row) : s(a), buf(of), rank(r)
    {
        width = shard_width(a, r);
        const uintptr_t at = uintptr_t(buf) + row * (a.ld ? a.ld : uint64_t(width)) * S;
        base = at & ~uintptr_t(15);
        shift = uint32_t(at & 15) / S;
        first = shift ? 1 : 0;
        end = max(first, (shift + width) / VEC);
    }
    // the access lies in the buffer
    __device__ __forceinline__ bool holds(const void *at, uint64_t bytes) const
    {
        return !kBoundsCheck || in_buffer(at, bytes, buf, shard_bytes(s, rank, S), s.status, s.site);
    }
    __device__ __forceinline__ bool holds_group(uint32_t j) const { return holds(group(j), 16); }
    __device__ __forceinline__ uint32_t head() const { return min(width, first * VEC - shift); }         // columns before the groups
    __device__ __forceinline__ uint32_t tail_begin() const { return head() + (end - first) * VEC; }      // first column after them
    __device__ __forceinline__ const void *group(uint32_t j) const { return reinterpret_cast<const void *>(base + uintptr_t(j) * 16); }
    __device__ __forceinline__ void *group_out(uint32_t j) const { return reinterpret_cast<void *>(base + uintptr_t(j) * 16); }
    __device__ __forceinline__ float column(uint32_t c) const
    {
        if (!holds(reinterpret_cast<const void *>(base + (uintptr_t(shift) + c) * S), S)) return 0.0f;
        return Traits<T>::load1(reinterpret_cast<const void *>(base), uint64_t(shift) + c);
    }
    __device__ __forceinline__ void set_column(uint32_t c, float v) const
    {
        if (!holds(reinterpret_cast<const void *>(base + (uintptr_t(shift) + c) * S), S)) return;
        Traits<T>::store1(reinterpret_cast<void *>(base), uint64_t(shift) + c, v);
    }
    // The edge column of thread t (or -1): t < VEC the head, the next VEC the tail.
    __device__ __forceinline__ int edge(uint32_t t, bool has_head, bool has_tail) const
    {
        if (has_head && t < head()) return int(t);
        if (has_tail && t >= VEC && t - VEC < width - tail_begin()) return int(tail_begin() + t - VEC);
        return -1;
    }
};

// Stores group j of the input row `in` to the same columns of `out`: one
// 128-bit store where both rows begin at the same place between boundaries.
template <typename T, int PM>
__device__ __forceinline__ void store_group(const ShardRow<T, PM> &out, const ShardRow<T, PM> &in, uint32_t j, const uint4 &v)
{
    using Tr = Traits<T>;
    if (out.shift == in.shift) {
        if (!out.holds_group(j)) return;
        st_stream_v4(out.group_out(j), v);
        return;
    }
    float f[Tr::VEC];
    Tr::unpack(v, f);
    const uint32_t c = j * Tr::VEC - in.shift;
#pragma unroll
    for (int i = 0; i < Tr::VEC; ++i) out.set_column(c + i, f[i]);
}

// Four words of -inf in the element type.
template <typename T>
__device__ __forceinline__ uint4 lowest_group()
{
    const uint32_t w = Traits<T>::VEC == 4 ? 0xff800000u : Traits<T>::kDtype == DT_BF16 ? 0xff80ff80u : 0xfc00fc00u;
    return make_uint4(w, w, w, w);
}

// ---------------------------------------------------------------------------
// Pairs of fp32 values, which sm_100 and later add and multiply in one
// instruction.
// ---------------------------------------------------------------------------

struct Pair {
    float x, y;
};

__device__ __forceinline__ Pair operator+(Pair a, Pair b)
{
    Pair r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b)
{
    Pair r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c)
{
    Pair r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// 2^x; results below the normal range are zero.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ Pair ex2(Pair v) { return {ex2(v.x), ex2(v.y)}; }

// The pairs of a group, the maximum of a group and a running one (a NaN is
// passed over), and a group from its pairs.
template <typename T>
struct Group;

template <>
struct Group<F32> {
    static constexpr int PAIRS = 2;
    using Max = float;
    __device__ static __forceinline__ Pair pair(const uint4 &v, int i)
    {
        return i == 0 ? Pair{__uint_as_float(v.x), __uint_as_float(v.y)} : Pair{__uint_as_float(v.z), __uint_as_float(v.w)};
    }
    __device__ static __forceinline__ Max lowest() { return -INFINITY; }
    __device__ static __forceinline__ Max max(Max m, const uint4 &v)
    {
        return fmaxf(m, fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w))));
    }
    __device__ static __forceinline__ float value(Max m) { return m; }
    __device__ static __forceinline__ uint4 pack(const Pair (&p)[2])
    {
        return make_uint4(__float_as_uint(p[0].x), __float_as_uint(p[0].y), __float_as_uint(p[1].x), __float_as_uint(p[1].y));
    }
};

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// 16-bit types compare two lanes at a time, in the type itself: widening keeps the order.
template <typename T, typename H2>
struct Group16 {
    static constexpr int PAIRS = 4;
    using Max = H2;
    __device__ static __forceinline__ H2 h2(uint32_t w) { return *reinterpret_cast<const H2 *>(&w); }
    __device__ static __forceinline__ Max lowest() { return h2(lowest_group<T>().x); }
    __device__ static __forceinline__ Max max(Max m, const uint4 &v)
    {
        return __hmax2(m, __hmax2(__hmax2(h2(v.x), h2(v.y)), __hmax2(h2(v.z), h2(v.w))));
    }
    __device__ static __forceinline__ uint4 pack(const Pair (&p)[4])
    {
        using Tr = Traits<T>;
        return make_uint4(Tr::pack2(p[0].x, p[0].y), Tr::pack2(p[1].x, p[1].y), Tr::pack2(p[2].x, p[2].y), Tr::pack2(p[3].x, p[3].y));
    }
};

template <>
struct Group<BF16> : Group16<BF16, __nv_bfloat162> {
    __device__ static __forceinline__ Pair pair(const uint4 &v, int i)
    {
        const uint32_t w = word(v, i);
        return {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
    }
    __device__ static __forceinline__ float value(Max m) { return fmaxf(__low2float(m), __high2float(m)); }
};

template <>
struct Group<F16> : Group16<F16, __half2> {
    __device__ static __forceinline__ Pair pair(const uint4 &v, int i)
    {
        const float2 f = __half22float2(h2(word(v, i)));
        return {f.x, f.y};
    }
    __device__ static __forceinline__ float value(Max m) { return fmaxf(__low2float(m), __high2float(m)); }
};

// A maximum of nothing but -inf: differences are formed against 0 instead, so
// that their exponentials are 0 and not NaN.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.0f : m; }

constexpr float kLog2e = 1.4426950408889634f;

template <int PM>
inline void fill_shards(Shards<PM> *s, const Launch &L, uint64_t rows, uint32_t vocab, uint64_t ld, unsigned site)
{
    const uint32_t p = uint32_t(L.p);
    for (uint32_t r = 0; r < p; ++r) {
        s->in[r] = L.src[r];
        s->out[r] = L.dst[r];
    }
    s->ld = ld;
    s->rows = rows;
    s->p = p;
    s->vocab = vocab;
    s->q = vocab / p;
    s->rem = vocab % p;
    s->by_q1 = fast_div(s->q + 1);
    s->by_q = fast_div(s->q ? s->q : 1);
    s->status = L.status;
    s->site = site;
    s->held = rows - (L.stall_test == 2 && rows ? 1 : 0);
}

// The most whole groups a row of the widest shard has.
template <typename T, int PM>
inline uint32_t widest_groups(const Shards<PM> &s) { return (s.q + (s.rem ? 1 : 0)) / Traits<T>::VEC; }

}  // namespace ccl
