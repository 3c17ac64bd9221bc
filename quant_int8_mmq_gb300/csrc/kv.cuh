// kv.cuh -- the 4-bit key/value cache: layout of a piece (one page of 64 tokens of one
// kv head), the widening of its codes, and the argument structures of its kernels.
//
// A group is 32 consecutive values of one head of one token.  Its scale s has 7
// significant bits, s in [2^-14, 896], and its codes n = 0..15 stand for s * (n - 8).
// 7 + 3 significant bits and a lowest bit of at least 2^-20 make every cached value
// exact in f16, so the attention kernels may feed the tensor cores f16 operands without
// a rounding on the cache's side.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>

#include "mmq.h"
#include "mmq_internal.h"
#include "ptx.cuh"

namespace mmq {

constexpr int KV_PAGE = MMQ_KV_PAGE;   // tokens per page
constexpr int KV_GROUP = 32;           // values per scale
constexpr int KV_PROMPT_ROWS = 256;    // rows of a kv_prompt.cu CTA
constexpr int KV_MAX_CLUSTER = 8;      // CTAs of a kv_step.cu cluster

// Byte offsets inside a piece of head size D; the documented layout is in mmq.h.
template <int D>
struct Piece {
    static_assert(D == 64 || D == 128, "head size");
    static constexpr int NG = D / KV_GROUP;
    static constexpr int K_CODES = 0;
    static constexpr int K_SCALES = 32 * D;
    static constexpr int V_CODES = 36 * D;
    static constexpr int V_SCALES = 68 * D;
    static constexpr int BYTES = 72 * D;

    // the 16-byte chunk that holds group g of token t's key
    __host__ __device__ static constexpr int k_chunk(int t, int g)
    {
        return K_CODES + t * (D / 2) + ((g ^ ((t >> (D == 128 ? 1 : 2)) & (NG - 1))) << 4);
    }
    __host__ __device__ static constexpr int k_scale(int t, int g) { return K_SCALES + (t * NG + g) * 2; }
    // the 16-byte chunk that holds values 16 a .. 16 a + 15 of the two tokens of pair p
    __host__ __device__ static constexpr int v_turn(int p)
    {
        return D == 128 ? ((p >> 2) ^ (p << 1 & 6)) & 7 : ((p >> 2) ^ (p & 2)) & 3;
    }
    __host__ __device__ static constexpr int v_chunk(int p, int a) { return V_CODES + p * D + ((a ^ v_turn(p)) << 4); }
    // the two f16 scales (tokens 2p, 2p + 1) of group g
    __host__ __device__ static constexpr int v_scale(int p, int g) { return V_SCALES + (p * NG + g) * 4; }
};

constexpr float KV_SCALE_MIN = 6.103515625e-05f;   // 2^-14
constexpr float KV_SCALE_MAX = 896.0f;             // 72 * 896 < 65504, the widening's addend

// A batch as the entry points describe it (mmq_kv_cache with its pointers typed).
struct KvView {
    uint8_t* pages;
    const int* table;
    const int* start;
    const int* length;
    int num_pages, kv_heads, batch, max_pages;
    unsigned int* bad;   // set to 1 when a table entry or a length leads outside the cache
};

struct KvRows {
    void* data;
    long long tok, head;   // strides in elements
};

// ------------------------------------------------------------------ widening
__device__ __forceinline__ uint32_t kv_h2u(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }
__device__ __forceinline__ __half2 kv_u2h(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }

// Pair I (0..3) of a code word w (the nibbles at bits 4 I and 4 I + 16), times the scale.
// A nibble at bits 0-3 under the exponent of 1024 reads 1024 + n, at bits 4-7 under that
// of 64 reads 64 + n.  The latter becomes s (n - 8) in one f16x2 fma with b = -72 s, of
// at most 11 significant bits; the former takes an add and a multiply, as 1032 s would
// be rounded.  Nothing is inexact.  Each mask and exponent is one three-input logic
// operation (written as such: as an expression it compiled to two, and the step kernel
// executed 555 of them a page for 314), and only pairs 2 and 3 share a shift, which
// keeps half of the work off the integer pipe.
__device__ __forceinline__ uint32_t kv_field(uint32_t x, uint32_t mask, uint32_t exponent)
{
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(exponent));   // (x & mask) | exponent
    return y;
}
template <int I>
__device__ __forceinline__ __half2 kv_widen(uint32_t w, __half2 s, __half2 b)
{
    const uint32_t x = I < 2 ? w : w >> 8;
    if constexpr (I % 2 == 0)
        return __hmul2(__hadd2(kv_u2h(kv_field(x, 0x000F000Fu, 0x64006400u)), __floats2half2_rn(-1032.0f, -1032.0f)), s);
    return __hfma2(kv_u2h(kv_field(x, 0x00F000F0u, 0x54005400u)), s, b);
}
__device__ __forceinline__ __half2 kv_addend(__half2 s) { return __hmul2(s, __floats2half2_rn(-72.0f, -72.0f)); }

// ------------------------------------------------------------------ rows of any type
template <typename T>
struct Elt;
template <>
struct Elt<float> {
    static __device__ __forceinline__ float to(float v) { return v; }
    static __device__ __forceinline__ float from(float v) { return v; }
};
template <>
struct Elt<__half> {
    static __device__ __forceinline__ float to(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half from(float v) { return __float2half_rn(v); }
};
template <>
struct Elt<__nv_bfloat16> {
    static __device__ __forceinline__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};

// Four consecutive elements; `wide` when their address is aligned to all four.
template <typename T>
__device__ __forceinline__ float4 load4(const T* p, bool wide)
{
    T e[4];
    if (wide) {
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(p);
        else
            *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            e[i] = p[i];
    }
    return make_float4(Elt<T>::to(e[0]), Elt<T>::to(e[1]), Elt<T>::to(e[2]), Elt<T>::to(e[3]));
}
// The same in two halves: the load, and the values once they are used.
template <typename T>
struct Raw4 {
    alignas(4 * sizeof(T)) T e[4];
    __device__ __forceinline__ void load(const T* p, bool wide)
    {
        if (wide) {
            if constexpr (sizeof(T) == 4)
                *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(p);
            else
                *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(p);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                e[i] = p[i];
        }
    }
    __device__ __forceinline__ float4 get() const
    {
        return make_float4(Elt<T>::to(e[0]), Elt<T>::to(e[1]), Elt<T>::to(e[2]), Elt<T>::to(e[3]));
    }
};
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v, bool wide)
{
    T e[4] = {Elt<T>::from(v.x), Elt<T>::from(v.y), Elt<T>::from(v.z), Elt<T>::from(v.w)};
    if (wide) {
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(e);
        else
            *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(e);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = e[i];
    }
}

__device__ __forceinline__ float kv_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// floor(log2 a) within [-126, 126], and 2^e there: scaling by them is exact, and a row
// whose largest magnitude is a comes to [1, 2), or to (0, 4) at the ends of the range.
__device__ __forceinline__ int kv_exponent(float a)
{
    return min(max(static_cast<int>(__float_as_uint(a) >> 23) - 127, -126), 126);
}
__device__ __forceinline__ float kv_pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// x = hi + lo in f16 (22 bits) for two values
__device__ __forceinline__ void kv_split2(float x, float y, uint32_t& hi, uint32_t& lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = kv_h2u(h);
    lo = kv_h2u(__floats2half2_rn(x - f.x, y - f.y));
}

// Softmax weights p = 2^(x - ref) are kept in f16 halves.  A fresh reference is `below` less
// than the row's largest x and stands until some x is 15 above it, so p is at most 2^15.  f16's
// least step is 2^-24: a weight may be off by 2^-25, which n keys together make n 2^-(25 + below)
// of the largest.  16-bit rows: 7, so that rows are rescaled rarely (by a factor of 2^8 or
// more); 131072 keys lose up to 3e-5, below the rounding of P.  f32 rows: 13, a factor of 4;
// 2^20 keys lose up to 4e-6 (with 7 a far tail of 131072 keys lost 6e-5).
template <typename T>
__host__ __device__ constexpr float kv_ref_below()
{
    return sizeof(T) == 4 ? 13.0f : 7.0f;
}
constexpr float KV_REF_LIMIT = 15.0f;

// Which keys of a page (64 from kbase on) a row at position pos sees, one bit each.
// Positions, windows and sinks stay below 2^30 (the entry point limits the latter two).
__device__ __forceinline__ uint64_t kv_seen_bits(int pos, int kbase, int window, int sinks)
{
    const int to = min(max(pos - kbase, -1), 63);
    uint64_t m = to < 0 ? 0 : ~0ull >> (63 - to);
    if (window > 0) {
        const int from = min(max(pos - window + 1 - kbase, 0), 64);
        const int sink = min(max(sinks - kbase, 0), 64);
        m &= (from < 64 ? ~0ull << from : 0) | (sink > 0 ? ~0ull >> (64 - sink) : 0);
    }
    return m;
}

// The sequence of packed row r: the last b with start[b] <= r, found by one warp, 32
// probes a step (sequences without rows are passed over).  0 <= result < batch whatever
// start holds.
__device__ __forceinline__ int kv_sequence_of(const int* start, int batch, int r, int lane)
{
    int lo = 0, n = batch;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool in = lane * step < n && (lane == 0 || start[i] <= r);
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, in));   // lane 0 is always in
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

// ------------------------------------------------------------------ launchers
// Lets `kernel` use `bytes` of dynamic shared memory, once per device (a bit of `done` each).
template <typename K>
cudaError_t kv_allow_smem(K* kernel, int bytes, std::atomic<uint64_t>* done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done->load(std::memory_order_acquire) & bit)
        return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        done->fetch_or(bit, std::memory_order_release);
    return e;
}

enum KvType { KV_F32 = 0, KV_F16 = 1, KV_BF16 = 2 };

cudaError_t launch_kv_write(const KvView& c, int dim, int dtype, const KvRows& k, const KvRows& v, bool wide,
                            int ntok, cudaStream_t s);
cudaError_t launch_kv_read(const KvView& c, int dim, int dtype, const KvRows& k, const KvRows& v, bool wide, int ntok,
                           cudaStream_t s);

// What an attention call computes; positions and lengths are read on the device.
struct AttendArgs {
    KvView c;
    KvRows q, out;
    int heads, group;      // group = heads / kv_heads
    int ntok;
    float scale_log2;      // softmax scale times log2(e)
    int window, sinks;
    int tile_rows;         // kv_step.cu: rows of a tile, 8 or (16-bit rows) 16
    int row_tiles;         // kv_step.cu: row tiles per (sequence, kv head); kv_prompt.cu: of the whole batch
    int nsplit;            // parts of the visible pages,
    int part_pages;        // each of so many
    int cluster;           // kv_step.cu: CTAs that share a part
    bool wide;
    float* part;           // nsplit > 1: [nsplit][ntok * heads][D] unnormalised sums
    float2* part_ml;       //             [nsplit][ntok * heads] {reference, sum}
    WaitCtl wc;
};

// The attention's last block (the others have a unit of work each): packed rows that no unit
// computes become zero, and are reported.  They are those before the first sequence's and past
// the last's, those of a sequence whose rows lead outside the packed ones, and those past the
// first `most` (new tokens times the group) of a sequence.  A block of its own keeps this off
// the others' time: as a branch of theirs it cost 64 single tokens and short prompts 1.3 %.
template <int D, typename T>
__device__ __forceinline__ void kv_clear_others(const AttendArgs& g, long long most)
{
    const long long n = g.ntok;
    // rows [lo, hi), counted through the group, of every kv head
    auto clear = [&](long long lo, long long hi) {
        if (threadIdx.x == 0)
            *g.c.bad = 1u;
        constexpr int FOURS = D / 4;
        for (int head = 0; head < g.heads; head += g.group) {
            if (g.nsplit > 1) {   // the join passes over parts without sums
                for (int split = 0; split < g.nsplit; ++split)
                    for (long long i = lo + threadIdx.x; i < hi; i += blockDim.x)
                        g.part_ml[(split * n + i / g.group) * g.heads + head + i % g.group] = make_float2(-INFINITY, 0.0f);
                continue;
            }
            for (long long i = lo * FOURS + threadIdx.x; i < hi * FOURS; i += blockDim.x) {
                const long long row = i / FOURS;
                store4(static_cast<T*>(g.out.data) + row / g.group * g.out.tok + (head + row % g.group) * g.out.head +
                           i % FOURS * 4,
                       make_float4(0.0f, 0.0f, 0.0f, 0.0f), g.wide);
            }
        }
    };
    for (int b0 = 0; b0 < g.c.batch; b0 += blockDim.x) {
        const int end = min(g.c.batch - b0, static_cast<int>(blockDim.x)) + b0;
        auto look = [&](int b, bool act) {
            const long long first = g.c.start[b], last = g.c.start[b + 1];
            const bool fits = first >= 0 && last >= first && last <= n;
            const bool before = b == 0 && first > 0, after = b == g.c.batch - 1 && last < n;
            const bool more = fits && (last - first) * g.group > most;
            if (act) {
                if (!fits)
                    clear(max(first, 0ll) * g.group, min(last, n) * g.group);
                if (before)
                    clear(0, min(first, n) * g.group);
                if (after)
                    clear(max(last, 0ll) * g.group, n * g.group);
                if (more)
                    clear(first * g.group + most, last * g.group);
            }
            return !fits || before || after || more;
        };
        const int b = b0 + static_cast<int>(threadIdx.x);
        if (!__syncthreads_or(b < end && look(b, false)))
            continue;
        for (int i = b0; i < end; ++i)
            look(i, true);
    }
}

struct AttendPlan {
    int kernel;      // 0: kv_step.cu, 1: kv_prompt.cu
    int tile_rows, row_tiles;
    int nsplit, part_pages, cluster;
    size_t part_bytes, ml_bytes;
};
AttendPlan plan_attend(int dtype, int heads, int kv_heads, int dim, int batch, int ntok, int max_q, int max_kv,
                       int max_pages, int window, int sinks);
cudaError_t launch_kv_step(const AttendArgs& a, int dim, int dtype, cudaStream_t s);
cudaError_t launch_kv_prompt(const AttendArgs& a, int dim, int dtype, cudaStream_t s);
cudaError_t launch_kv_join(const AttendArgs& a, int dim, int dtype, cudaStream_t s);

}  // namespace mmq
