// kv_rows.cuh -- rows on their way into and out of the 4-bit cache: a token's place, eight
// values of a lane, and their codes.  A lane holds 8 consecutive values of a key or a value row,
// 4 lanes a group of 32.
#pragma once

#include "kv.cuh"

namespace mmq {

// Offset of the page of packed row r in the pool, and its slot there; -1 (and the cache's
// error word set) when the row has no place in the cache.
__device__ __forceinline__ long long kv_page_of(const KvView& c, int r, long long page_bytes, int lane, int* slot)
{
    const int b = kv_sequence_of(c.start, c.batch, r, lane);
    const int first = c.start[b], end = c.start[b + 1];
    const long long pos = static_cast<long long>(c.length[b]) - end + r;
    if (r >= first && r < end && pos >= 0 && pos < static_cast<long long>(c.max_pages) * KV_PAGE) {
        const int page = c.table[static_cast<size_t>(b) * c.max_pages + static_cast<size_t>(pos / KV_PAGE)];
        if (page >= 0 && page < c.num_pages) {
            *slot = static_cast<int>(pos % KV_PAGE);
            return page * page_bytes;
        }
    }
    if (lane == 0)
        *c.bad = 1u;
    *slot = 0;
    return -1;
}

// How a warp's lanes share the rows of a head: LANES lanes a row, keys then values.
template <int D>
struct Share {
    static constexpr int LANES = D / 8;
    static constexpr int HEADS = 32 / (2 * LANES);   // heads at once
};

// Eight elements from p on; `wide` when p is aligned to 16 bytes.
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool wide, float (&x)[8])
{
    T e[8];
    if (wide) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
            reinterpret_cast<uint4*>(e)[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = Elt<T>::to(e[i]);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, bool wide, const float (&x)[8])
{
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        e[i] = Elt<T>::from(x[i]);
    if (wide) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
            reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<uint4*>(e)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[i] = e[i];
    }
}

// x / y rounded to nearest, r being 1 / y rounded to nearest: the quotient's error, exact in
// an fma, corrects it (P. Markstein, IBM J. Res. Dev. 34, 1990).  Where the error underflows
// the quotient is far below every rounding boundary used here.
__device__ __forceinline__ float quotient(float x, float y, float r)
{
    const float q = x * r;
    return fmaf(fmaf(-q, y, x), r, q);
}

// The scale of a group whose largest magnitude is a.
__device__ __forceinline__ float kv_scale(float a)
{
    const float amax = fminf(a, 1e30f);   // the scale's limit is far below
    const uint32_t up = (__float_as_uint(quotient(amax, 7.5f, 1.0f / 7.5f)) + 0x1FFFFu) & ~0x1FFFFu;
    return fminf(fmaxf(__uint_as_float(up), KV_SCALE_MIN), KV_SCALE_MAX);
}
// code = rint(x / s) + 8 in the low bits of 1.5 * 2^23 + 8 + x / s; limiting x to [-8 s, 7 s]
// limits the rounded quotient to [-8, 7]
template <int N>
__device__ __forceinline__ void kv_codes(const float (&x)[N], float s, uint32_t (&n)[N])
{
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < N; ++i)
        n[i] = __float_as_uint(quotient(fminf(fmaxf(x[i], -8.0f * s), 7.0f * s), s, inv) + 12582920.0f);
}

// The codes of a lane's 8 values of a key or a value row: two 16-bit halves, and the group's scale.
// The four lanes of a group call it together.
struct Codes8 {
    uint32_t lo, hi;
    float s;
};
__device__ __forceinline__ Codes8 kv_quantise8(float (&x)[8], bool key)
{
    float a = 0.0f;
    bool odd = false;   // some x is no number
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a = fmaxf(a, fabsf(x[i]));
        odd |= x[i] != x[i];
    }
    if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = x[i] == x[i] ? x[i] : 0.0f;
    }
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
    const float s = kv_scale(a);
    uint32_t n[8];
    kv_codes(x, s, n);
    // 16-bit halves of four codes: key values 0 2 4 6 | 1 3 5 7, value values 0 1 2 3 | 4 5 6 7
    const uint32_t lo = n[0] + ((key ? n[2] : n[1]) << 4) + ((key ? n[4] : n[2]) << 8) + ((key ? n[6] : n[3]) << 12);
    const uint32_t hi = (key ? n[1] : n[4]) + ((key ? n[3] : n[5]) << 4) + ((key ? n[5] : n[6]) << 8) + (n[7] << 12);
    return {lo, hi, s};
}

// Where a lane's codes and its group's scale lie in a piece: lane l of a row's D/8, in slot `slot`.
template <int D>
struct Place8 {
    int codes, scale;
    __device__ __forceinline__ Place8(int slot, int l, bool key)
        : codes(key ? Piece<D>::k_chunk(slot, l / 4) + l % 4 * 4
                    : Piece<D>::v_chunk(slot / 2, l / 2) + l % 2 * 8 + slot % 2 * 2),
          scale(key ? Piece<D>::k_scale(slot, l / 4) : Piece<D>::v_scale(slot / 2, l / 4) + slot % 2 * 2)
    {
    }
    __device__ __forceinline__ void put(uint8_t* piece, const Codes8& c, int l, bool key) const
    {
        if (key) {
            *reinterpret_cast<uint32_t*>(piece + codes) = __byte_perm(c.lo, c.hi, 0x5410);
        } else {
            *reinterpret_cast<uint16_t*>(piece + codes) = static_cast<uint16_t>(c.lo);
            *reinterpret_cast<uint16_t*>(piece + codes + 4) = static_cast<uint16_t>(c.hi);
        }
        if (l % 4 == 0)
            *reinterpret_cast<__half*>(piece + scale) = __float2half_rn(c.s);   // exact
    }
};

}  // namespace mmq
