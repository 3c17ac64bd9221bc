// kv_cache.cu -- writing new tokens into the 4-bit key/value cache, and reading it back.
//
// A group of 32 values gets s = the least number of 7 significant bits that is at least
// amax / 7.5 (so 7.5 s covers the largest value and rounding moves no value by more than
// s / 2), kept within [2^-14, 896], and codes rint(x / s) limited to -8..7.  Both
// divisions are IEEE: as s has 7 bits, (k + 1/2) s is exact in f32 and a quotient rounds
// to k + 1/2 only if x equals it, so the codes are the nearest ones, ties to even, and do
// not depend on how the work is laid out.
//
// Both kernels move bytes.  A lane holds 8 consecutive values of a key or a value row
// (one code word of a key), a warp the key and the value of one head (two heads of 64),
// so rows move as 16-byte accesses in whole lines and a group's largest magnitude is two
// shuffles among its 4 lanes; a warp keeps its token and walks over heads, which shares
// the search for the token's place.  The 8 warps of a CTA hold consecutive tokens, whose
// value codes share their sectors.
//
// On GB300: reading 121318 tokens of 8 heads of 128 as bf16 takes 111 us (5.8 TB/s, a copy
// reaches 6.8); writing 3314 f32 tokens of 32 heads of 128 and reading them back 56 us
// (4.4 TB/s), of which the write is a little under half and bound by its instructions; the read
// waits for its loads and the queue of its stores, in 2.2 rounds of CTAs.
#include "kv.cuh"

namespace mmq {
namespace {

constexpr int WARPS = 8;

// Offset of the page of packed row r in the pool, and its slot there; -1 (and the cache's
// error word set) when the row has no place in the cache.
__device__ __forceinline__ long long page_of(const KvView& c, int r, long long page_bytes, int lane, int* slot)
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

// x / y rounded to nearest, r being 1 / y rounded to nearest: the quotient's error, exact in
// an fma, corrects it (P. Markstein, IBM J. Res. Dev. 34, 1990).  Where the error underflows
// the quotient is far below every rounding boundary used here.
__device__ __forceinline__ float quotient(float x, float y, float r)
{
    const float q = x * r;
    return fmaf(fmaf(-q, y, x), r, q);
}

template <int D, typename T>
__global__ void __launch_bounds__(WARPS * 32) kv_write_kernel(const KvView c, const KvRows k, const KvRows v, bool wide,
                                                              int ntok, int heads_a_warp)
{
    using P = Piece<D>;
    constexpr int LANES = Share<D>::LANES;
    const int r = blockIdx.x * WARPS + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (r >= ntok)
        return;
    grid_dep_wait();
    grid_dep_launch();
    const long long page_bytes = static_cast<long long>(c.kv_heads) * P::BYTES;
    int slot;
    const long long page = page_of(c, r, page_bytes, lane, &slot);
    const int l = lane % LANES;
    const bool key = lane / LANES % 2 == 0;
    const int h0 = blockIdx.y * heads_a_warp, h1 = min(c.kv_heads, h0 + heads_a_warp);
    const KvRows& in = key ? k : v;
    const T* row = static_cast<const T*>(in.data) + r * in.tok + 8 * l;
    // this lane's codes and its group's scale in a piece
    const int codes = key ? P::k_chunk(slot, l / 4) + l % 4 * 4 : P::v_chunk(slot / 2, l / 2) + l % 2 * 8 + slot % 2 * 2;
    const int scale = key ? P::k_scale(slot, l / 4) : P::v_scale(slot / 2, l / 4) + slot % 2 * 2;
    uint8_t* pages = c.pages + page;
    float ahead[8];   // the next head's values, on their way
    load8(row + min(h0 + lane / (2 * LANES), h1 - 1) * in.head, wide, ahead);
    for (int h = h0; h < h1; h += Share<D>::HEADS) {
        const int head = h + lane / (2 * LANES);
        const bool mine = head < h1;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = ahead[i];
        if (h + Share<D>::HEADS < h1)
            load8(row + min(head + Share<D>::HEADS, h1 - 1) * in.head, wide, ahead);
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
        const float amax = fminf(a, 1e30f);   // the scale's limit is far below
        const uint32_t up = (__float_as_uint(quotient(amax, 7.5f, 1.0f / 7.5f)) + 0x1FFFFu) & ~0x1FFFFu;
        const float s = fminf(fmaxf(__uint_as_float(up), KV_SCALE_MIN), KV_SCALE_MAX);
        const float inv = __frcp_rn(s);
        // code = rint(x / s) + 8 in the low bits of 1.5 * 2^23 + 8 + x / s; limiting x to [-8 s, 7 s]
        // limits the rounded quotient to [-8, 7]
        uint32_t n[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            n[i] = __float_as_uint(quotient(fminf(fmaxf(x[i], -8.0f * s), 7.0f * s), s, inv) + 12582920.0f);
        // 16-bit halves of four codes: key values 0 2 4 6 | 1 3 5 7, value values 0 1 2 3 | 4 5 6 7
        const uint32_t lo = n[0] + ((key ? n[2] : n[1]) << 4) + ((key ? n[4] : n[2]) << 8) + ((key ? n[6] : n[3]) << 12);
        const uint32_t hi = (key ? n[1] : n[4]) + ((key ? n[3] : n[5]) << 4) + ((key ? n[5] : n[6]) << 8) + (n[7] << 12);
        if (!mine || page < 0)
            continue;
        uint8_t* piece = pages + head * P::BYTES;
        if (key) {
            *reinterpret_cast<uint32_t*>(piece + codes) = __byte_perm(lo, hi, 0x5410);
        } else {
            *reinterpret_cast<uint16_t*>(piece + codes) = static_cast<uint16_t>(lo);
            *reinterpret_cast<uint16_t*>(piece + codes + 4) = static_cast<uint16_t>(hi);
        }
        if (l % 4 == 0)
            *reinterpret_cast<__half*>(piece + scale) = __float2half_rn(s);   // exact
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, bool wide, const __half2 (&x)[4])
{
    T e[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(x[i]);
        e[2 * i] = Elt<T>::from(f.x);
        e[2 * i + 1] = Elt<T>::from(f.y);
    }
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

template <int D, typename T>
__global__ void __launch_bounds__(WARPS * 32) kv_read_kernel(const KvView c, const KvRows k, const KvRows v, bool wide,
                                                             int ntok, int heads_a_warp)
{
    using P = Piece<D>;
    constexpr int LANES = Share<D>::LANES;
    const int r = blockIdx.x * WARPS + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (r >= ntok)
        return;
    grid_dep_wait();
    grid_dep_launch();
    const long long page_bytes = static_cast<long long>(c.kv_heads) * P::BYTES;
    int slot;
    const long long page = page_of(c, r, page_bytes, lane, &slot);
    const int l = lane % LANES;
    const bool key = lane / LANES % 2 == 0;
    const int h0 = blockIdx.y * heads_a_warp, h1 = min(c.kv_heads, h0 + heads_a_warp);
    const KvRows& out = key ? k : v;
    T* row = static_cast<T*>(out.data) + r * out.tok + 8 * l;
    const int codes = key ? P::k_chunk(slot, l / 4) + l % 4 * 4 : P::v_chunk(slot / 2, l / 2) + l % 2 * 8;
    const int scale = key ? P::k_scale(slot, l / 4) : P::v_scale(slot / 2, l / 4) + slot % 2 * 2;
    const uint32_t half = slot % 2 ? 0x7632 : 0x5410;   // this token's 16 bits of each word
    const uint8_t* pages = c.pages + max(page, 0ll);
    // a batch's loads are all in flight before its first store
    constexpr int BATCH = 4;
    const int step = Share<D>::HEADS, next = key ? 4 : 8;
    for (int h = h0 + lane / (2 * LANES); h < h1; h += BATCH * step) {
        uint32_t z0[BATCH], z1[BATCH];
        __half2 s[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (page < 0 || h + i * step >= h1)
                continue;
            const uint8_t* piece = pages + (h + i * step) * P::BYTES;
            if (key) {
                z0[i] = *reinterpret_cast<const unsigned int*>(piece + codes);
            } else {
                const uint2 w = *reinterpret_cast<const uint2*>(piece + codes);   // both tokens'
                z0[i] = w.x;
                z1[i] = w.y;
            }
            s[i] = __half2half2(__ushort_as_half(*reinterpret_cast<const unsigned short*>(piece + scale)));
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (h + i * step >= h1)
                break;
            __half2 x[4];
            if (page >= 0) {
                // pairs 0 and 1 at nibble 0 and the next (key) or the one after (value) of z0, 2 and 3 of z1
                if (key) {
                    z1[i] = z0[i] >> 8;
                } else {   // this token's half of each word, beside itself moved by a value
                    const uint32_t m = __byte_perm(z0[i], z1[i], half);
                    z0[i] = __byte_perm(m, m >> 4, 0x5410);
                    z1[i] = __byte_perm(m, m >> 4, 0x7632);
                }
                x[0] = kv_widen<0>(z0[i], s[i], s[i]);
                x[1] = kv_widen<0>(z0[i] >> next, s[i], s[i]);
                x[2] = kv_widen<0>(z1[i], s[i], s[i]);
                x[3] = kv_widen<0>(z1[i] >> next, s[i], s[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[j] = __floats2half2_rn(0.0f, 0.0f);
            }
            store8(row + (h + i * step) * out.head, wide, x);
        }
    }
}

template <int D, typename T>
cudaError_t launch_rows(bool write, const KvView& c, const KvRows& k, const KvRows& v, bool wide, int ntok,
                        cudaStream_t s)
{
    // a warp takes more heads of its token once every SM has its 64 warps
    const long long spread = static_cast<long long>(ntok) * c.kv_heads / (152 * 64);
    int heads = static_cast<int>(spread < 1 ? 1 : spread > 8 ? 8 : spread);
    heads = (heads + Share<D>::HEADS - 1) / Share<D>::HEADS * Share<D>::HEADS;
    const dim3 grid((ntok + WARPS - 1) / WARPS, (c.kv_heads + heads - 1) / heads);
    count_launch();
    if (write)
        return launch_dependent(kv_write_kernel<D, T>, grid, dim3(WARPS * 32), s, c, k, v, wide, ntok, heads);
    return launch_dependent(kv_read_kernel<D, T>, grid, dim3(WARPS * 32), s, c, k, v, wide, ntok, heads);
}

template <int D>
cudaError_t launch_rows(bool write, const KvView& c, int dtype, const KvRows& k, const KvRows& v, bool wide, int ntok,
                        cudaStream_t s)
{
    return dtype == KV_F32   ? launch_rows<D, float>(write, c, k, v, wide, ntok, s)
           : dtype == KV_F16 ? launch_rows<D, __half>(write, c, k, v, wide, ntok, s)
                             : launch_rows<D, __nv_bfloat16>(write, c, k, v, wide, ntok, s);
}

}  // namespace

cudaError_t launch_kv_write(const KvView& c, int dim, int dtype, const KvRows& k, const KvRows& v, bool wide, int ntok,
                            cudaStream_t s)
{
    return dim == 128 ? launch_rows<128>(true, c, dtype, k, v, wide, ntok, s)
                      : launch_rows<64>(true, c, dtype, k, v, wide, ntok, s);
}

cudaError_t launch_kv_read(const KvView& c, int dim, int dtype, const KvRows& k, const KvRows& v, bool wide, int ntok,
                           cudaStream_t s)
{
    return dim == 128 ? launch_rows<128>(false, c, dtype, k, v, wide, ntok, s)
                      : launch_rows<64>(false, c, dtype, k, v, wide, ntok, s);
}

}  // namespace mmq
