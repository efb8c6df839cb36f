// Rank buffers that hold the shards of [rows, vocab] logits: rank r has the
// columns of balanced chunk r (the library's chunks: the larger ones first),
// row-major with a row stride of its own.
//
// A row is worked through in 16-byte groups that lie on 16-byte boundaries of
// memory wherever the row itself begins: group j of a row that begins s
// elements past a boundary holds columns [j*VEC - s, (j+1)*VEC - s).  Groups
// that lie wholly inside the row are moved with one 128-bit access, the ones
// at its two ends element by element, so odd vocabularies, odd strides and
// unaligned shards run at the speed of aligned ones.  Every rank has the same
// number nv of group slots (enough for the widest shard at the worst s), so
// that slot i of a row belongs to rank i / nv; slots past a row's end hold
// nothing.
#pragma once

#include "device.cuh"

namespace ccl {

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
    uint32_t nv;        // group slots per rank
    FastDiv by_nv, by_q1, by_q;
    unsigned *status;   // the communicator's status block (checked build)
};

template <int PM>
__device__ __forceinline__ uint32_t shard_width(const Shards<PM> &a, uint32_t r) { return a.q + (r < a.rem ? 1u : 0u); }
template <int PM>
__device__ __forceinline__ uint32_t shard_begin(const Shards<PM> &a, uint32_t r) { return r * a.q + min(r, a.rem); }

template <int PM>
__device__ __forceinline__ uint32_t rank_of_slot(const Shards<PM> &a, uint32_t slot)
{
    return PM == 1 ? 0u : div_by(slot, a.by_nv);
}

template <int PM>
__device__ __forceinline__ uint32_t rank_of_token(const Shards<PM> &a, uint32_t v)
{
    if constexpr (PM == 1) return 0u;
    const uint32_t big = a.rem * (a.q + 1);
    return v < big ? div_by(v, a.by_q1) : a.rem + div_by(v - big, a.by_q);
}

// One row of one shard.
struct ShardRow {
    uintptr_t base;    // the 16-byte boundary at or below the row's first element
    uint32_t shift;    // elements between the boundary and the row
    uint32_t width;
};

template <typename T>
__device__ __forceinline__ ShardRow shard_row(const void *buf, uint64_t ld, uint64_t row, uint32_t width)
{
    constexpr uint32_t S = 16 / Traits<T>::VEC;
    const uintptr_t at = uintptr_t(buf) + row * (ld ? ld : uint64_t(width)) * S;
    return {at & ~uintptr_t(15), uint32_t(at & 15) / S, width};
}

// Columns [e, e + VEC) of group j; e may be negative, and the end past the row.
template <typename T>
__device__ __forceinline__ int group_begin(const ShardRow &r, uint32_t j) { return int(j * Traits<T>::VEC) - int(r.shift); }

template <typename T>
__device__ __forceinline__ bool group_whole(const ShardRow &r, int e) { return e >= 0 && uint32_t(e) + Traits<T>::VEC <= r.width; }

// Group j's values; columns outside the row read as -inf.
template <typename T>
__device__ __forceinline__ uint4 load_group(const ShardRow &r, uint32_t j, bool row_ok, unsigned *status, unsigned site)
{
    using Tr = Traits<T>;
    const int e = group_begin<T>(r, j);
    if (group_whole<T>(r, e) && in_bounds(row_ok, status, site, j))
        return ld_coherent_v4(reinterpret_cast<const void *>(r.base + uintptr_t(j) * 16));
    float f[Tr::VEC];
#pragma unroll
    for (int i = 0; i < Tr::VEC; ++i) {
        const bool in = e + i >= 0 && uint32_t(e + i) < r.width;
        f[i] = in && in_bounds(row_ok, status, site, j) ? Tr::load1(reinterpret_cast<const void *>(r.base), uint64_t(j) * Tr::VEC + i)
                                                        : -INFINITY;
    }
    return Tr::pack(f);
}

// Stores the columns of input group j (input row `in`) to the same columns of
// the output row: whole groups with one 128-bit store where both rows begin
// at the same place between boundaries.
template <typename T>
__device__ __forceinline__ void store_group(const ShardRow &out, const ShardRow &in, uint32_t j, const uint4 &v, bool row_ok,
                                            unsigned *status, unsigned site)
{
    using Tr = Traits<T>;
    const int e = group_begin<T>(in, j);
    if (out.shift == in.shift && group_whole<T>(in, e)) {
        if (in_bounds(row_ok, status, site, j)) st_stream_v4(reinterpret_cast<void *>(out.base + uintptr_t(j) * 16), v);
        return;
    }
    float f[Tr::VEC];
    Tr::unpack(v, f);
#pragma unroll
    for (int i = 0; i < Tr::VEC; ++i)
        if (e + i >= 0 && uint32_t(e + i) < in.width && in_bounds(row_ok, status, site, j))
            Tr::store1(reinterpret_cast<void *>(out.base), uint64_t(out.shift) + uint64_t(e + i), f[i]);
}

// 2^x; results below the normal range are zero.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// Host: fills everything but the pointers' aliases checks have established.
template <int PM>
inline void fill_shards(Shards<PM> *s, const Launch &L, uint64_t rows, uint32_t vocab, uint64_t ld)
{
    const uint32_t p = uint32_t(L.p), es = uint32_t(elem_bytes(L.dtype)), vec = 16 / es;
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
    const uint32_t wide = s->q + (s->rem ? 1 : 0);
    bool aligned = true;
    for (uint32_t r = 0; r < p; ++r) {
        const uint64_t stride = (ld ? ld : s->q + (r < s->rem ? 1 : 0)) * es;
        aligned = aligned && uintptr_t(L.src[r]) % 16 == 0 && (rows == 1 || stride % 16 == 0);
    }
    s->nv = (wide + (aligned ? 0 : vec - 1) + vec - 1) / vec;
    s->by_nv = fast_div(s->nv);
    s->by_q1 = fast_div(s->q + 1);
    s->by_q = fast_div(s->q ? s->q : 1);
    s->status = L.status;
}

}  // namespace ccl
