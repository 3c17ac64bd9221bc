// kv_cache.cu -- writing new tokens into the 4-bit key/value cache, and reading it back.
//
// A group of 32 values gets s = the least number of 7 significant bits that is at least
// amax / 7.5 (so 7.5 s covers the largest value and rounding moves no value by more than
// s / 2), kept within [2^-14, 896], and codes rint(x / s) limited to -8..7.  Both
// divisions are IEEE: as s has 7 bits, (k + 1/2) s is exact in f32 and a quotient rounds
// to k + 1/2 only if x equals it, so the codes are the nearest ones, ties to even, and do
// not depend on how the work is laid out.
//
// Both kernels move bytes: a warp takes one (token, head), each lane four values, so
// that rows are read and written in whole 128-byte lines.  Writing, a group's largest
// magnitude is three shuffles within its 8 lanes.
#include "kv.cuh"

namespace mmq {
namespace {

constexpr int WARPS = 8;

// The piece and slot of packed row r and one head; piece null (and the cache's error word
// set) when the row has no place in the cache.
template <int D>
__device__ __forceinline__ uint8_t* piece_of(const KvView& c, int r, int head, int lane, int* slot)
{
    const int b = kv_sequence_of(c.start, c.batch, r, lane);
    const int first = c.start[b], end = c.start[b + 1];
    const long long pos = static_cast<long long>(c.length[b]) - end + r;
    if (r >= first && r < end && pos >= 0 && pos < static_cast<long long>(c.max_pages) * KV_PAGE) {
        const int page = c.table[static_cast<size_t>(b) * c.max_pages + static_cast<size_t>(pos / KV_PAGE)];
        if (page >= 0 && page < c.num_pages) {
            *slot = static_cast<int>(pos % KV_PAGE);
            return c.pages + (static_cast<size_t>(page) * c.kv_heads + head) * Piece<D>::BYTES;
        }
    }
    if (lane == 0)
        *c.bad = 1u;
    *slot = 0;
    return nullptr;
}

__device__ __forceinline__ uint32_t code_of(float x, float s)
{
    const float y = x == x ? rintf(__fdiv_rn(x, s)) : 0.0f;
    return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(y, -8.0f), 7.0f)) + 8);
}

// Codes and scale of this lane's four values; every 8 lanes hold one group.
__device__ __forceinline__ void quantise(float4 x, uint32_t (&n)[4], __half* scale)
{
    float a = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
    for (int d = 1; d < 8; d <<= 1)
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    const uint32_t up = (__float_as_uint(__fdiv_rn(a, 7.5f)) + 0x1FFFFu) & ~0x1FFFFu;
    const float s = fminf(fmaxf(__uint_as_float(up), KV_SCALE_MIN), KV_SCALE_MAX);
    n[0] = code_of(x.x, s);
    n[1] = code_of(x.y, s);
    n[2] = code_of(x.z, s);
    n[3] = code_of(x.w, s);
    *scale = __float2half_rn(s);   // exact
}

// Lane l of a head holds values 4l .. 4l + 3.  (u, p, h) of value 8u + 2p + h: an even lane
// has p = 0, 1 of its word, the odd lane after it p = 2, 3.
template <int D>
__device__ __forceinline__ void put_key(uint8_t* piece, int slot, int l, float4 x)
{
    uint32_t n[4];
    __half s;
    quantise(x, n, &s);
    const uint32_t part = n[0] | n[1] << 16 | n[2] << 4 | n[3] << 20;
    const uint32_t odd = __shfl_down_sync(0xffffffffu, part, 1);
    if (piece == nullptr)
        return;
    if (l % 2 == 0)
        *reinterpret_cast<uint32_t*>(piece + Piece<D>::k_chunk(slot, l / 8) + (l % 8) * 2) = part | odd << 8;
    if (l % 8 == 0)
        *reinterpret_cast<__half*>(piece + Piece<D>::k_scale(slot, l / 8)) = s;
}

template <int D>
__device__ __forceinline__ void put_value(uint8_t* piece, int slot, int l, float4 x)
{
    uint32_t n[4];
    __half s;
    quantise(x, n, &s);
    if (piece == nullptr)
        return;
    const int pair = slot / 2, e = slot % 2;
    *reinterpret_cast<uint16_t*>(piece + Piece<D>::v_chunk(pair, l / 4) + (l % 4) * 4 + e * 2) =
        static_cast<uint16_t>(n[0] | n[1] << 4 | n[2] << 8 | n[3] << 12);
    if (l % 8 == 0)
        *reinterpret_cast<__half*>(piece + Piece<D>::v_scale(pair, l / 8) + e * 2) = s;
}

template <int D, typename T>
__global__ void __launch_bounds__(WARPS * 32) kv_write_kernel(const KvView c, const KvRows k, const KvRows v, bool wide,
                                                              long long units)
{
    const long long u = static_cast<long long>(blockIdx.x) * WARPS + threadIdx.x / 32;
    if (u >= units)
        return;
    const int lane = threadIdx.x % 32;
    const int r = static_cast<int>(u / c.kv_heads), head = static_cast<int>(u % c.kv_heads);
    const T* kr = static_cast<const T*>(k.data) + r * k.tok + head * k.head;
    const T* vr = static_cast<const T*>(v.data) + r * v.tok + head * v.head;
    int slot;
    if constexpr (D == 128) {
        const float4 x = load4(kr + 4 * lane, wide), y = load4(vr + 4 * lane, wide);
        uint8_t* piece = piece_of<D>(c, r, head, lane, &slot);
        put_key<D>(piece, slot, lane, x);
        put_value<D>(piece, slot, lane, y);
    } else {   // the lower half of the warp takes the key, the upper half the value
        const float4 x = load4((lane < 16 ? kr : vr) + 4 * (lane % 16), wide);
        uint8_t* piece = piece_of<D>(c, r, head, lane, &slot);
        put_key<D>(lane < 16 ? piece : nullptr, slot, lane % 16, x);
        put_value<D>(lane < 16 ? nullptr : piece, slot, lane % 16, x);
    }
}

// Code n of scale s; the difference and the product are exact.
__device__ __forceinline__ float value_of(uint32_t n, float s) { return s * (static_cast<float>(n & 15u) - 8.0f); }

template <int D>
__device__ __forceinline__ float4 get_key(const uint8_t* piece, int slot, int l)
{
    const uint32_t w = *reinterpret_cast<const uint32_t*>(piece + Piece<D>::k_chunk(slot, l / 8) + (l % 8 / 2) * 4) >>
                       (l % 2 * 8);
    const float s = __half2float(*reinterpret_cast<const __half*>(piece + Piece<D>::k_scale(slot, l / 8)));
    return make_float4(value_of(w, s), value_of(w >> 16, s), value_of(w >> 4, s), value_of(w >> 20, s));
}
template <int D>
__device__ __forceinline__ float4 get_value(const uint8_t* piece, int slot, int l)
{
    const int pair = slot / 2, e = slot % 2;
    const uint32_t w =
        *reinterpret_cast<const uint16_t*>(piece + Piece<D>::v_chunk(pair, l / 4) + (l % 4) * 4 + e * 2);
    const float s = __half2float(*reinterpret_cast<const __half*>(piece + Piece<D>::v_scale(pair, l / 8) + e * 2));
    return make_float4(value_of(w, s), value_of(w >> 4, s), value_of(w >> 8, s), value_of(w >> 12, s));
}

template <int D, typename T>
__global__ void __launch_bounds__(WARPS * 32) kv_read_kernel(const KvView c, const KvRows k, const KvRows v, bool wide,
                                                             long long units)
{
    const long long u = static_cast<long long>(blockIdx.x) * WARPS + threadIdx.x / 32;
    if (u >= units)
        return;
    const int lane = threadIdx.x % 32;
    const int r = static_cast<int>(u / c.kv_heads), head = static_cast<int>(u % c.kv_heads);
    T* kr = static_cast<T*>(k.data) + r * k.tok + head * k.head;
    T* vr = static_cast<T*>(v.data) + r * v.tok + head * v.head;
    int slot;
    const uint8_t* piece = piece_of<D>(c, r, head, lane, &slot);
    const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if constexpr (D == 128) {
        store4(kr + 4 * lane, piece ? get_key<D>(piece, slot, lane) : none, wide);
        store4(vr + 4 * lane, piece ? get_value<D>(piece, slot, lane) : none, wide);
    } else {
        const int l = lane % 16;
        const float4 x = piece == nullptr ? none : lane < 16 ? get_key<D>(piece, slot, l) : get_value<D>(piece, slot, l);
        store4((lane < 16 ? kr : vr) + 4 * l, x, wide);
    }
}

template <int D, typename T>
cudaError_t launch_rows(bool write, const KvView& c, const KvRows& k, const KvRows& v, bool wide, int ntok,
                        cudaStream_t s)
{
    const long long units = static_cast<long long>(ntok) * c.kv_heads;
    const unsigned int blocks = static_cast<unsigned int>((units + WARPS - 1) / WARPS);
    count_launch();
    if (write)
        kv_write_kernel<D, T><<<blocks, WARPS * 32, 0, s>>>(c, k, v, wide, units);
    else
        kv_read_kernel<D, T><<<blocks, WARPS * 32, 0, s>>>(c, k, v, wide, units);
    return cudaGetLastError();
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
