// kv_weigh.cu -- the weight that each key of the 4-bit cache receives from the new tokens' rows:
//
//   out[j] = decay in[j] (tokens that were there) + sum over rows 2^(x_j - ref) / sum,
//   x_j = scale log2(e) q . k_j
//
// with each row's reference and sum from the attention that ran before (f32, so its own division by
// the sum and this one agree; the sum over rows is f32 too, in a fixed order, without atomics).
//
// Three ways, the first two chosen by the scores' size, the third by the rows' number:
//
// kv_finish_weights_kernel (few rows: the step kernel ran).  The attention has left its scores, 4 bytes
// a row and key, so that K is not read and widened again: for a token on 131071 keys, 32 heads on 8,
// 56 us with the attention (47.5 alone) for 78 with the next kernel; 64 sequences of up to 8192, 113 for 165.
// Where scores would take more than a gigabyte the next kernel runs (more sizes at weigh_plan).
//
// kv_weigh_few_kernel (up to 128 rows per sequence and kv head) and kv_weigh_many_kernel (more):
// S^T = K Q^T on the tensor cores.  Keys are the 128 lanes of tensor memory and rows its columns, so a
// key's sum over the rows stays in a thread's registers (many rows: four threads') and nothing is added
// up across CTAs; what a column needs (coefficient, reference, 1 / sum) is read by whole warps at once.  K is widened to f16,
// exactly, from the codes; rows are scaled by a power of two and, where they are f32, split in two f16
// parts.  With few rows these stay in shared memory and the keys stream by; with many, 256 keys
// stay and the rows stream by.
//
// What bounds them: the sums.  Few rows: a warpgroup's loop of load from tensor memory, wait, constants and
// exponentials (cycles below); 32 f16 tokens on 131072 keys, 32 heads on 8, 67 us of 147 (1.1 TB/s of K).
// Many rows: an exponential and two fma an element, and three reads of a column's constants for every four
// elements of two keys.  2 x 2048 f16 tokens of 32 heads on 8 on 16384 keys 640 us, with the rows' laying
// out, beside 816 for the attention.  Without its exponentials an earlier form of the kernel took
// 13 % less, without the constants' reads 20 %; those could go into the product (three more values of every
// row), but an argument that is far from 0 costs weights three bits, and rows of a tile need one factor.
#include <cfloat>
#include <type_traits>

#include "kv.cuh"

namespace mmq {
namespace {

constexpr int KEYS = 128;       // lanes of tensor memory
constexpr int MOST_ROWS = 128;  // columns of a step

// What a row's column needs, in shared memory and (many rows) in the workspace.
struct alignas(16) Columns {
    float coef[MOST_ROWS], minus[MOST_ROWS], inv[MOST_ROWS];   // minus the reference
    int pos[MOST_ROWS];
};

__device__ __forceinline__ bool wait(const WeighArgs& w, uint32_t bar, uint32_t parity)
{
    return mbar_wait_asleep(bar, parity, w.a.wc.limit_ns, w.a.wc.err);
}
// All lanes ask the same barrier in one instruction, so the warp stays together: with lanes that
// waited for different barriers, or one for all, it came apart, and tcgen05's .aligned
// instructions after that faulted.
__device__ __forceinline__ bool warp_wait(const WeighArgs& w, uint32_t bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, wait(w, bar, parity));
}

// The sequence and kv head that a CTA works on.
struct Unit {
    int b, head;
    int first, rows;        // packed rows; rows counted through the group
    int length, pos0;       // tokens; position of the first new one
    int plo, phi;           // positions of the first and last row
    const int* table;
};
__device__ __forceinline__ bool unit_of(const WeighArgs& w, int b, int head, Unit& u)
{
    const AttendArgs& g = w.a;
    u.head = head;
    u.b = b;
    u.first = g.c.start[u.b];
    const int last = g.c.start[u.b + 1];
    if (u.first < 0 || last <= u.first || last > g.ntok)
        return false;
    const int new_tokens = last - u.first, counted = min(new_tokens, w.max_q);
    if (new_tokens > counted)
        *g.c.bad = 1u;
    u.rows = counted * g.group;
    u.length = min(max(g.c.length[u.b], 0), g.c.max_pages * KV_PAGE);
    u.pos0 = max(g.c.length[u.b], 0) - new_tokens;
    u.plo = u.pos0;
    u.phi = u.pos0 + counted - 1;
    u.table = g.c.table + static_cast<size_t>(u.b) * g.c.max_pages;
    return true;
}

// Whether a row sees any of the keys [k0, k0 + n), and whether all see all.
__device__ __forceinline__ bool any_seen(const AttendArgs& g, int plo, int phi, int k0, int n)
{
    return k0 <= phi && (g.window == 0 || k0 + n - 1 > plo - g.window || k0 < g.sinks);
}
__device__ __forceinline__ bool all_seen(const AttendArgs& g, int plo, int phi, int k0, int n)
{
    return k0 + n - 1 <= plo && (g.window == 0 || k0 > phi - g.window || k0 + n <= g.sinks);
}

// The codes of one key, on their way into an operand tile.
template <int D>
struct KeyCodes {
    uint4 code[D / 32];
    uint2 scale;
    // of slot `slot` of a piece; one that is not there gives zeros: any code times the scale 0
    __device__ __forceinline__ void get(const uint8_t* src, int slot, bool there)
    {
        using P = Piece<D>;
        scale = make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            code[i] = make_uint4(0, 0, 0, 0);
        if (!there)
            return;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            code[i] = *reinterpret_cast<const uint4*>(src + P::k_chunk(slot, i));
        if constexpr (D == 128)
            scale = *reinterpret_cast<const uint2*>(src + P::k_scale(slot, 0));
        else
            scale.x = *reinterpret_cast<const uint32_t*>(src + P::k_scale(slot, 0));
    }
    // the 32 values of a group as 16 pairs
    __device__ __forceinline__ void widen(int gr, uint32_t (&o)[16]) const
    {
        const uint32_t both = gr < 2 ? scale.x : scale.y;
        const __half2 s = kv_u2h(__byte_perm(both, 0, gr % 2 ? 0x3232 : 0x1010)), sb = kv_addend(s);
        const uint32_t v[4] = {code[gr].x, code[gr].y, code[gr].z, code[gr].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[4 * i] = kv_h2u(kv_widen<0>(v[i], s, sb));
            o[4 * i + 1] = kv_h2u(kv_widen<1>(v[i], s, sb));
            o[4 * i + 2] = kv_h2u(kv_widen<2>(v[i], s, sb));
            o[4 * i + 3] = kv_h2u(kv_widen<3>(v[i], s, sb));
        }
    }
    // row t of [64-value block][128 keys] tiles, 128-byte swizzle
    __device__ __forceinline__ void widen(uint8_t* dst, int t) const
    {
#pragma unroll
        for (int gr = 0; gr < D / 32; ++gr) {
            uint32_t o[16];
            widen(gr, o);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4*>(dst + gr / 2 * KEYS * 128 + t * 128 + ((gr % 2 * 4 + i) ^ (t & 7)) * 16) =
                    make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
    }
};

// One row, four values a lane, as operand row r (modulo 8) at dst, its 64-value blocks `block` bytes
// apart, by a warp, an f32 row's low part `low` bytes on; the coefficient that makes its products powers of two.
template <int D, typename T>
__device__ __forceinline__ float put_row(const AttendArgs& g, float4 x, uint8_t* dst, size_t block, int r, size_t low, int lane)
{
    float a = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    const int e = kv_exponent(a);
    const float f = kv_pow2(-e);
    if (lane < D / 4) {
        uint2 hi, lo;
        kv_split2(x.x * f, x.y * f, hi.x, lo.x);
        kv_split2(x.z * f, x.w * f, hi.y, lo.y);
        const int d = 4 * lane;
        uint8_t* at = dst + d / 64 * block + ((d / 8 % 8 ^ (r & 7)) << 4) + d % 8 * 2;
        *reinterpret_cast<uint2*>(at) = hi;
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<uint2*>(at + low) = lo;   // a multiple of 8 rows: the same turn
    }
    return fminf(fmaxf(g.scale_log2 * kv_pow2(e), 1e-38f), 1e38f);
}

// The rows of a unit, warp `warp` of `warps` taking every warps-th, four loads on their way at once.
template <int D, typename T>
__device__ __forceinline__ void put_rows(const AttendArgs& g, const Unit& u, int n, int warp, int warps, uint8_t* dst,
                                         Columns* cols, int lane)
{
    constexpr int BATCH = 4;
    const int rows = min(u.rows, n);
    for (int r0 = warp; r0 < n; r0 += BATCH * warps) {
        Raw4<T> x[BATCH];
        float2 stats[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = r0 + i * warps;
            stats[i] = make_float2(0.0f, 0.0f);
            if (r < rows) {
                const long long token = u.first + r / g.group;
                const int h = u.head * g.group + r % g.group;
                stats[i] = g.stats[token * g.heads + h];
                if (lane < D / 4)
                    x[i].load(static_cast<const T*>(g.q.data) + token * g.q.tok + h * g.q.head + 4 * lane, g.wide);
            }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = r0 + i * warps;
            if (r >= n)
                break;
            const bool there = stats[i].y > 0.0f && lane < D / 4;   // a row without weights is given as zeros
            const float coef = put_row<D, T>(g, there ? x[i].get() : make_float4(0.0f, 0.0f, 0.0f, 0.0f), dst + r * 128,
                                             (sizeof(T) == 4 ? 2 : 1) * n * 128, r, n * 128, lane);
            if (lane == 0) {
                cols->coef[r] = coef;
                cols->minus[r] = -stats[i].x;
                cols->inv[r] = stats[i].y;
                cols->pos[r] = r < rows ? u.pos0 + r / g.group : -1;
            }
        }
    }
}

// K Q^T of one step: 128 keys by n rows.
template <int D, int PARTS>
__device__ __forceinline__ void product(uint32_t lead, uint32_t to, uint32_t k, uint32_t q, int q_block, uint32_t idesc)
{
    constexpr int KB = D / 64;
#pragma unroll
    for (int part = PARTS - 1; part >= 0; --part)   // lo first, while the sums, cut toward zero, are small
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const uint64_t a = sdesc_k_sw128(k + kb * KEYS * 128);
            const uint64_t b = sdesc_k_sw128(q + (part * KB + kb) * q_block);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                umma_f16_by(lead, to, a + 2u * kk, b + 2u * kk, idesc, (part < PARTS - 1 || kb || kk) ? 1u : 0u);
        }
}

// A warp has what it wants of S.
__device__ __forceinline__ void release(uint32_t bar, int lane)
{
    tc_fence_before();
    __syncwarp();
    if (lane == 0)
        mbar_arrive(bar);
}

// What four columns need.  Asked for before a load from tensor memory is waited for: behind the wait it
// would be another latency.
struct Four {
    float4 coef, minus, inv;
    __device__ __forceinline__ void load(const Columns* cols, int c)
    {
        coef = *reinterpret_cast<const float4*>(cols->coef + c);
        minus = *reinterpret_cast<const float4*>(cols->minus + c);
        inv = *reinterpret_cast<const float4*>(cols->inv + c);
    }
};
template <int N>
struct Constants {
    Four four[N / 4];
    __device__ __forceinline__ Constants(const Columns* cols, int c)
    {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            four[i].load(cols, c + 4 * i);
    }
};

// The weights of some columns, c0 on, of KS keys (key, key + KEYS, ...).  MASKED: those from n on and those
// that do not see the key count nothing.
template <bool MASKED, int N, int KS>
__device__ __forceinline__ void add_columns(const AttendArgs& g, const float (&x)[KS][N], const Constants<N>& at, const Columns* cols,
                                            int c0, int n, int key, float2 (&sum)[KS])
{
#pragma unroll
    for (int c = 0; c < N; c += 4) {
        if (MASKED && c0 + c >= n)
            break;
        const float4 f = at.four[c / 4].coef, r = at.four[c / 4].minus, v = at.four[c / 4].inv;
        const int4 pos = MASKED ? *reinterpret_cast<const int4*>(cols->pos + c0 + c) : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const float2 a = ffma2(make_float2(x[k][c], x[k][c + 1]), make_float2(f.x, f.y), make_float2(r.x, r.y));
            const float2 b = ffma2(make_float2(x[k][c + 2], x[k][c + 3]), make_float2(f.z, f.w), make_float2(r.z, r.w));
            float4 p = make_float4(kv_ex2(a.x), kv_ex2(a.y), kv_ex2(b.x), kv_ex2(b.y));
            if constexpr (MASKED) {
                const int j = key + k * KEYS;
                auto seen = [&](int i, int at) {
                    return c0 + c + i < n && j <= at && (g.window == 0 || j > at - g.window || j < g.sinks);
                };
                p.x = seen(0, pos.x) ? p.x : 0.0f;
                p.y = seen(1, pos.y) ? p.y : 0.0f;
                p.z = seen(2, pos.z) ? p.z : 0.0f;
                p.w = seen(3, pos.w) ? p.w : 0.0f;
            }
            sum[k] = ffma2(make_float2(p.x, p.y), make_float2(v.x, v.y), sum[k]);
            sum[k] = ffma2(make_float2(p.z, p.w), make_float2(v.z, v.w), sum[k]);
        }
    }
}

// ------------------------------------------------------------------ few rows
// One CTA an SM; all tiles of 128 keys, sequence by sequence and head by head, are cut into even
// shares, so that lengths may differ as they like and a CTA's pipeline runs on from one head to
// the next.  What a tile costs its warps is a chain of dependent instructions, waits among them,
// longer than the 400 cycles that its bytes take: so each role is several warpgroups' or warps', which
// take the tiles in turn.  Clock stamps of one CTA, 131072 keys, means of 40 tiles, 128 / 64 / 32 columns of
// f16 rows: codes widened 810 / 850 / 860 cycles; product issued to S seen 1400 / 1500 / 1610; sums 4270 / 2430 /
// 1550, of which S is free again after 3650 / 1830 / 970; a tile every 1890 / 1280 / 1000.  With 128
// columns that is one group's S: awaited, read and given back in 5600 cycles, a third of which is a
// tile's share; the widening groups and the issuing warp wait for it.  With fewer columns no role is
// busy all the time: what is left are the handoffs between them.
constexpr int GROUPS = 3, ROW_WARPS = 4, COPY_WARPS = 2;
constexpr int SUM_WARP = 4 * GROUPS, ROW_WARP = SUM_WARP + 4 * GROUPS, COPY_WARP = ROW_WARP + ROW_WARPS,
              MMA_WARP = COPY_WARP + COPY_WARPS, FEW_WARPS = MMA_WARP + 1, FEW_THREADS = FEW_WARPS * 32;
constexpr int BATCH = 4;               // tiles a copying warp asks for at once

// K as an operand lies in tensor memory: widened codes go there from registers, and neither they
// nor the products' reading of them take shared memory's bandwidth (in shared memory a tile
// took 1000 cycles, most of them that).
//
// Waits tell one round of a barrier from the next by its parity, so nobody may wait for a round
// while the one before it is open.  Each warpgroup has a buffer of its own (S, and K unless two
// have to do), and one warp issues all products in order: a group that has its buffer back
// from step i knows that all steps before i are done with, and the stages of codes are more than
// the steps that can be open.
constexpr int MAX_Q = 2, MAX_STAGES = 16;
static_assert(MAX_STAGES % (BATCH * COPY_WARPS) == 0, "stages");
enum { F_RFULL = 0, F_REMPTY = F_RFULL + MAX_STAGES, F_KFULL = F_REMPTY + MAX_STAGES, F_KEMPTY = F_KFULL + GROUPS,
       F_SFULL = F_KEMPTY + GROUPS, F_SEMPTY = F_SFULL + GROUPS, F_QFULL = F_SEMPTY + GROUPS, F_QEMPTY = F_QFULL + MAX_Q,
       F_DRAIN = F_QEMPTY + MAX_Q, F_BARS };

// Where everything is in shared memory, and how many buffers of each there are.
struct FewLayout {
    int qbufs, kbufs, stages, stage_bits, columns;   // operands Q and K, codes on their way (a power of two: a
                                                     // division took as long as the rest of a step), columns of S
    int ring, cols, ids, bars, bytes;
};

template <int D, typename T>
struct Few {
    static constexpr int PARTS = sizeof(T) == 4 ? 2 : 1, KB = D / 64;
    static constexpr int K_COLUMNS = D / 2;
    static constexpr int HALF = Piece<D>::V_CODES, STAGE = 2 * HALF;    // a page's keys, a step's
    static constexpr int q_bytes(int n) { return PARTS * KB * n * 128; }
    // low parts of f32 rows: n more columns of S, or, where that is too many, a second product
    __host__ __device__ static constexpr bool side_by_side(int n) { return PARTS * n <= 128; }
    static FewLayout layout(int n)
    {
        FewLayout l = {};
        const int wide = side_by_side(n) ? PARTS * n : n;
        l.columns = wide <= 32 ? 32 : wide <= 64 ? 64 : 128;
        l.kbufs = GROUPS * (l.columns + K_COLUMNS) <= 512 ? GROUPS : 2;
        for (l.qbufs = MAX_Q;; --l.qbufs) {
            l.cols = l.qbufs * q_bytes(n);
            l.ids = l.cols + l.qbufs * static_cast<int>(sizeof(Columns));
            l.bars = l.ids + MAX_STAGES * 8;
            l.ring = (l.bars + F_BARS * 8 + 15) / 16 * 16;
            // a multiple of the copying warps' turns, so that a stage is always filled by the same lanes
            constexpr int TURN = BATCH * COPY_WARPS;
            const int left = (225 * 1024 - l.ring) / STAGE / TURN * TURN;
            l.stages = left < MAX_STAGES ? left : MAX_STAGES;
            l.bytes = l.ring + l.stages * STAGE + 1024;   // and the alignment
            l.stage_bits = l.stages == 16 ? 4 : 3;
            if (l.stages > 0 || l.qbufs == 1)
                return l;
        }
    }
};
static_assert(GROUPS * MOST_ROWS + 2 * Few<128, float>::K_COLUMNS <= 512, "tensor memory");

// A run of one head's tiles [t0, t1); the n of them of which some row sees a key are the first n1
// (before the window) and those from `second` on.
struct Run {
    int t0, t1, n1, n, second;
    __device__ __forceinline__ int tile(int i) const { return i < n1 ? t0 + i : second + i - n1; }
};

// The tiles [c, end) of all sequences' and heads' as runs, each role on its own.
struct Walk {
    const WeighArgs& w;
    Unit u;
    int b, head, tiles, tile;   // of the current sequence; first tile of the next run
    long long left;
    __device__ __forceinline__ Walk(const WeighArgs& args, int b0, long long skip, long long count) : w(args), b(b0), left(count)
    {
        open();
        head = tiles ? static_cast<int>(skip / tiles) : 0;
        tile = tiles ? static_cast<int>(skip % tiles) : 0;
    }
    static __device__ __forceinline__ int tiles_of(const WeighArgs& w, int b)
    {
        const int first = w.a.c.start[b], last = w.a.c.start[b + 1];
        const int length = min(max(w.a.c.length[b], 0), w.a.c.max_pages * KV_PAGE);
        return first < 0 || last <= first || last > w.a.ntok ? 0 : (length + KEYS - 1) / KEYS;
    }
    __device__ __forceinline__ void open()
    {
        tiles = 0;
        while (left > 0 && (tiles = tiles_of(w, b)) == 0)
            ++b;
        if (tiles)
            unit_of(w, b, 0, u);
    }
    // false at the end
    __device__ __forceinline__ bool next(Run& r)
    {
        if (left <= 0)
            return false;
        if (tile == tiles) {
            tile = 0;
            if (++head == w.a.c.kv_heads) {
                head = 0;
                ++b;
                open();
            }
        }
        u.head = head;
        r.t0 = tile;
        r.t1 = static_cast<int>(min(static_cast<long long>(tiles), tile + left));
        left -= r.t1 - r.t0;
        tile = r.t1;
        // tile t is seen if t KEYS <= phi and, with a window, t KEYS + KEYS - 1 > plo - window or t KEYS < sinks
        const AttendArgs& g = w.a;
        const int end = min(r.t1, u.phi < 0 ? 0 : u.phi / KEYS + 1);
        const int from = g.window > 0 ? max(u.plo - g.window + 1, 0) / KEYS : 0;
        const int sinks = min((g.sinks + KEYS - 1) / KEYS, from);
        r.n1 = max(min(end, sinks) - r.t0, 0);
        r.second = max(r.t0, from);
        r.n = r.n1 + max(end - r.second, 0);
        return true;
    }
};

// A ring's place and the parity of its round.
struct Turn {
    int i = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void next(int n)
    {
        if (++i == n) {
            i = 0;
            round ^= 1u;
        }
    }
};

__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

template <int D, typename T>
__global__ void __launch_bounds__(FEW_THREADS, 1) kv_weigh_few_kernel(const WeighArgs w, const FewLayout l)
{
    using C = Few<D, T>;
    using P = Piece<D>;
    const AttendArgs& g = w.a;
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long total, skip;
    __shared__ long long warp_sum[FEW_WARPS];
    __shared__ int first_b;
    __shared__ uint32_t tmem_at;
    const uint32_t raw = smem_u32(smem_raw), pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t sbase = raw + pad;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    auto bar = [&](int i) -> uint32_t { return sbase + static_cast<uint32_t>(l.bars) + 8u * static_cast<uint32_t>(i); };
    Columns* cols = reinterpret_cast<Columns*>(smem + l.cols);
    int2* ids = reinterpret_cast<int2*>(smem + l.ids);

    if (threadIdx.x == 0) {
        for (int i = 0; i < MAX_STAGES; ++i) {
            mbar_init(bar(F_RFULL + i), 1);
            mbar_init(bar(F_REMPTY + i), 4);
        }
        for (int i = 0; i < GROUPS; ++i) {
            mbar_init(bar(F_KFULL + i), 4);
            mbar_init(bar(F_KEMPTY + i), 1);
            mbar_init(bar(F_SFULL + i), 1);
            mbar_init(bar(F_SEMPTY + i), 4);
        }
        for (int i = 0; i < MAX_Q; ++i) {
            mbar_init(bar(F_QFULL + i), ROW_WARPS);
            mbar_init(bar(F_QEMPTY + i), 1 + 4 * GROUPS);
        }
        mbar_init(bar(F_DRAIN), 1);
        fence_barrier_init();
        total = 0;
    }
    grid_dep_wait();
    // this CTA's share of all tiles: where it begins
    long long sum = 0;
    for (int b = threadIdx.x; b < g.c.batch; b += FEW_THREADS)
        sum += Walk::tiles_of(w, b);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0)
        warp_sum[warp] = sum;
    __syncthreads();
    long long all = 0;
    for (int i = 0; i < FEW_WARPS; ++i)
        all += warp_sum[i];
    all *= g.c.kv_heads;
    const long long c0 = all * blockIdx.x / gridDim.x, c1 = all * (blockIdx.x + 1) / gridDim.x;
    if (c0 == c1)
        return;
    for (int b0 = 0; b0 < g.c.batch; b0 += FEW_THREADS) {
        const int b = b0 + threadIdx.x;
        const long long mine = b < g.c.batch ? static_cast<long long>(Walk::tiles_of(w, b)) * g.c.kv_heads : 0;
        long long to = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, to, d);
            to += lane >= d ? v : 0;
        }
        __syncthreads();   // the sums of the round before are read
        if (lane == 31)
            warp_sum[warp] = to;
        __syncthreads();
        to += total;
        for (int i = 0; i < warp; ++i)
            to += warp_sum[i];
        if (to - mine <= c0 && c0 < to) {
            first_b = b;
            skip = c0 - (to - mine);
        }
        __syncthreads();
        if (threadIdx.x == FEW_THREADS - 1)
            total = to;
    }
    if (warp == MMA_WARP) {
        tmem_alloc(smem_u32(&tmem_at), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at;
    const int n = w.cols, q_bytes = C::PARTS * C::KB * n * 128;
    Walk walk(w, first_b, skip, c1 - c0);
    const Unit& u = walk.u;
    Run run;
    bool ok = true;
    // the first run's rows: by all, but the warps that copy, which have begun
    if (warp < COPY_WARP) {
        walk.u.head = walk.head;
        put_rows<D, T>(g, u, n, warp, COPY_WARP, smem, cols, lane);
        fence_proxy_async_smem();
        named_bar_sync(1, COPY_WARP * 32);
    }

    if (warp < SUM_WARP) {
        // ------------------------------------------------------------ widening
        const int t = threadIdx.x % KEYS, group = warp / 4;
        const uint32_t k_at = tmem + GROUPS * l.columns + group * C::K_COLUMNS + (static_cast<uint32_t>(t & ~31) << 16);
        int step = 0, turn = group, visit = 0;   // of the run's first seen tile; steps until the group's next; its steps
        if (group >= l.kbufs)
            ok = false;   // two groups have to do
        while (ok && walk.next(run)) {
            for (; turn < run.n; turn += l.kbufs, ++visit) {
                const int at = step + turn, stage = at & (l.stages - 1);
                ok = warp_wait(w, bar(F_KEMPTY + group), (visit & 1) ^ 1) && warp_wait(w, bar(F_RFULL + stage), at >> l.stage_bits & 1);
                if (!ok)
                    break;
                tc_fence_after();
                const int2 page = ids[stage];
                KeyCodes<D> codes;
                codes.get(smem + l.ring + stage * C::STAGE + t / KV_PAGE * C::HALF, t % KV_PAGE,
                          (t < KV_PAGE ? page.x : page.y) >= 0);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(F_REMPTY + stage));
#pragma unroll
                for (int gr = 0; gr < D / 32; ++gr) {
                    uint32_t v[16];
                    codes.widen(gr, v);
                    tmem_store16(k_at + 16 * gr, v);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(F_KFULL + group));
            }
            turn -= run.n;
            step += run.n;
        }
    } else if (warp < ROW_WARP) {
        // ------------------------------------------------------------ sums: a thread a key
        const int group = (warp - SUM_WARP) / 4, t = threadIdx.x % KEYS;
        const uint32_t s_at = tmem + group * l.columns + (static_cast<uint32_t>(t & ~31) << 16);
        const bool still = w.in == w.out && w.decay == 1.0f, both = C::PARTS == 2 && C::side_by_side(n);
        const size_t page_floats = static_cast<size_t>(g.c.kv_heads) * KV_PAGE;
        int turn = group, visit = 0;   // steps until the group's next; its steps
        Turn q;
        while (ok && walk.next(run)) {
            const int rows = min(u.rows, n);
            const float* in = w.in + u.head * KV_PAGE + t % KV_PAGE;
            float* out = w.out + u.head * KV_PAGE + t % KV_PAGE;
            // the page of this thread's key of a tile, if the pool has it
            auto page_of = [&](int tile) {
                const int key = tile * KEYS + t;
                const int page = key < u.length ? u.table[key / KV_PAGE] : -1;
                return page < g.c.num_pages ? page : -1;
            };
            auto had = [&](int page, int tile) { return page >= 0 && tile * KEYS + t < u.pos0 ? in[page * page_floats] : 0.0f; };
            // tiles without a key that is seen; with decay 1 in place nothing changes but for new tokens
            for (int tile = still ? max(run.t0, max(u.pos0, 0) / KEYS) : run.t0; tile < run.t1; ++tile) {
                if (tile < run.t0 + run.n1 || (tile >= run.second && tile < run.second + run.n - run.n1) || tile % GROUPS != group)
                    continue;
                const int page = page_of(tile);
                if (page >= 0)
                    out[page * page_floats] = w.decay * had(page, tile);
                else if (tile * KEYS + t < u.length)
                    *g.c.bad = 1u;
            }
            // what a key had, and the page of the one after, are on their way while a tile is added up
            int i = turn, page = -1, page1 = -1;
            float old = 0.0f;
            if (i < run.n) {
                page = page_of(run.tile(i));
                if (i + GROUPS < run.n)
                    page1 = page_of(run.tile(i + GROUPS));
                old = had(page, run.tile(i));
            }
            ok = warp_wait(w, bar(F_QFULL + q.i), q.round);
            for (; ok && i < run.n; i += GROUPS, ++visit) {
                const int tile = run.tile(i), key = tile * KEYS + t;
                const bool more = i + GROUPS < run.n;
                const float old1 = more ? had(page1, run.tile(i + GROUPS)) : 0.0f;
                const int page2 = i + 2 * GROUPS < run.n ? page_of(run.tile(i + 2 * GROUPS)) : -1;
                ok = warp_wait(w, bar(F_SFULL + group), visit & 1);
                if (!ok)
                    break;
                tc_fence_after();
                const bool plain = all_seen(g, u.plo, u.phi, tile * KEYS, KEYS);   // columns past the rows are zeros
                float2 got[1] = {make_float2(0.0f, 0.0f)};
                auto add = [&](const float (&x)[1][8], const Constants<8>& at, int c) {
                    if (plain)
                        add_columns<false>(g, x, at, cols + q.i, c, rows, key, got);
                    else
                        add_columns<true>(g, x, at, cols + q.i, c, rows, key, got);
                };
                for (int c = 0; c < rows; c += both ? 8 : 16) {
                    const Constants<8> at(cols + q.i, c);
                    float x[1][8], y[1][8];   // 8 columns and their low parts, or the 8 after them
                    tmem_ld8x2_wait(s_at + c, s_at + c + (both ? n : 8), x[0], y[0]);
                    if (c + (both ? 8 : 16) >= rows)
                        release(bar(F_SEMPTY + group), lane);
                    if (both) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            x[0][j] += y[0][j];
                    }
                    add(x, at, c);
                    if (!both)
                        add(y, Constants<8>(cols + q.i, c + 8), c + 8);
                }
                if (page >= 0)
                    out[page * page_floats] = (key < u.pos0 ? w.decay * old : 0.0f) + (got[0].x + got[0].y);
                page = page1;
                page1 = page2;
                old = old1;
            }
            turn = i - run.n;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(F_QEMPTY + q.i));
            q.next(l.qbufs);
        }
    } else if (warp < COPY_WARP) {
        // ------------------------------------------------------------ rows
        Turn q;
        for (bool first = true; ok && walk.next(run); first = false) {
            if (!first) {
                ok = warp_wait(w, bar(F_QEMPTY + q.i), q.round ^ 1u);
                if (!ok)
                    break;
                put_rows<D, T>(g, u, n, warp - ROW_WARP, ROW_WARPS, smem + q.i * q_bytes, cols + q.i, lane);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(F_QFULL + q.i));
            q.next(l.qbufs);
        }
    } else if (warp < MMA_WARP) {
        // ------------------------------------------------------------ codes
        // two lanes a tile, one for each of its pages
        const int mine = lane / 2 % BATCH, half = lane % 2;
        const bool act_lane = lane < 2 * BATCH;
        int step = 0;       // of the run's first seen tile
        uint32_t asked = 0, odd = 0;    // bit s: this lane has filled stage s; in an odd round last
        while (ok && walk.next(run)) {
            auto id_of = [&](int i) {
                const int p = 2 * run.tile(i) + half;
                return act_lane && i < run.n && p * KV_PAGE < u.length ? u.table[p] : -1;
            };
            // batches are counted over all runs, so that the warps take turns
            const int from = step / BATCH;
            auto base_of = [&](int batch) { return (from + batch) * BATCH - step; };   // the batch's first tile in the run
            int batch = (from % COPY_WARPS == warp - COPY_WARP) ? 0 : 1;
            int page = base_of(batch) + mine >= 0 ? id_of(base_of(batch) + mine) : -1;
            for (; base_of(batch) < run.n; batch += COPY_WARPS) {
                const int i = base_of(batch) + mine;
                const int page_next = id_of(base_of(batch + COPY_WARPS) + mine);
                const bool act = act_lane && i >= 0 && i < run.n;
                if (page >= g.c.num_pages || (page < 0 && act && (2 * run.tile(i) + half) * KV_PAGE < u.length)) {
                    *g.c.bad = 1u;
                    page = -1;
                }
                const int at = (step + max(i, 0)) & (l.stages - 1);
                const uint32_t round = (step + max(i, 0)) >> l.stage_bits & 1;
                ok = __all_sync(0xffffffffu, !act || wait(w, bar(F_REMPTY + at), round ^ 1u));
                if (!ok)
                    break;
                const int other = __shfl_xor_sync(0xffffffffu, page, 1);
                if (act && half == 0) {
                    ids[at] = make_int2(page, other);
                    mbar_arrive_expect_tx(bar(F_RFULL + at), ((page >= 0) + (other >= 0)) * C::HALF);
                    asked |= 1u << at;
                    odd = (odd & ~(1u << at)) | round << at;
                }
                __syncwarp();
                if (act && page >= 0) {
                    fence_proxy_async_smem();   // the stage was read with ordinary loads
                    bulk_g2s(sbase + l.ring + at * C::STAGE + half * C::HALF,
                             g.c.pages + (static_cast<size_t>(page) * g.c.kv_heads + u.head) * P::BYTES, C::HALF,
                             bar(F_RFULL + at));
                }
                page = page_next;
            }
            step += run.n;
        }
        // the last fill of each stage lands before the CTA ends
        for (int s = 0; s < l.stages; ++s)
            if (asked >> s & 1u)
                mbar_drain_wait(bar(F_RFULL + s), odd >> s & 1u, WAIT_LIMIT_NS, g.wc.err);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ products
        const uint32_t lead = elect_one();
        const bool both = C::PARTS == 2 && C::side_by_side(n);
        const uint32_t idesc = idesc_f16_f32(KEYS, both ? 2 * n : n);
        const int block = C::PARTS * n * 128;
        Turn q, k, s;
        while (ok && walk.next(run)) {
            ok = warp_wait(w, bar(F_QFULL + q.i), q.round);
            const uint32_t rows = sbase + q.i * q_bytes;
            for (int i = 0; ok && i < run.n; ++i) {
                ok = warp_wait(w, bar(F_KFULL + k.i), k.round) && warp_wait(w, bar(F_SEMPTY + s.i), s.round ^ 1u);
                if (!ok)
                    break;
                tc_fence_after();
                // lo first, while the sums, cut toward zero, are small
                for (int part = C::PARTS == 1 || both ? 0 : 1; part >= 0; --part)
#pragma unroll
                    for (int kb = 0; kb < C::KB; ++kb) {
                        const uint64_t b = sdesc_k_sw128(rows + kb * block + part * n * 128);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f16_ts_by(lead, tmem + s.i * l.columns,
                                           tmem + GROUPS * l.columns + k.i * C::K_COLUMNS + 32 * kb + 8 * kk,
                                           b + 2u * kk, idesc, (kb || kk || (C::PARTS == 2 && !both && part == 0)) ? 1u : 0u);
                    }
                umma_commit_by(lead, bar(F_SFULL + s.i));
                umma_commit_by(lead, bar(F_KEMPTY + k.i));
                k.next(l.kbufs);
                s.next(GROUPS);
            }
            if (ok)
                umma_commit_by(lead, bar(F_QEMPTY + q.i));
            q.next(l.qbufs);
        }
        umma_commit_by(lead, bar(F_DRAIN));
        if (lead)
            mbar_drain_wait(bar(F_DRAIN), 0, WAIT_LIMIT_NS, g.wc.err);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == MMA_WARP)
        tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ many rows
// Rows as operands in the workspace: [kv head][part][64-value block][row], and [kv head][row] coefficients.
// Those of sequence b begin at first_row(b), on a multiple of 8, where the swizzle's turn begins, so that a
// step's 128 rows are one copy a block from wherever it begins.  From one sequence that has rows to the
// next both its slot and its first token grow by one at least, so the lesser of them tells their rows
// apart.  (In tiles of 128 rows a sequence, a batch of single tokens and one long prompt took up to 16 times the room.)
//
// A step: 128 rows by both halves of the keys, into one of two pairs of buffers.  The columns of the rows,
// of which a warp makes what the sums need out of the attention's results, are kept four steps, as the
// sums are behind the products.  In place of one of 256 keys a CTA could take more, and wait less for its
// start (9600 cycles of a CTA's 28000 for a prompt of 3314), but a prompt's first keys are seen by all rows
// and its last by few, and small pieces, the long ones first, even that out.
template <int D, typename T>
struct Many {
    static constexpr int PARTS = sizeof(T) == 4 ? 2 : 1, KB = D / 64;
    static constexpr int BLOCK = MOST_ROWS * 128;
    static constexpr int Q_BYTES = PARTS * KB * BLOCK;
    static constexpr int K_BYTES = KB * KEYS * 128;        // of 128 keys
    static constexpr int STAGES = 2, CSTAGES = 4;          // operands, columns on their way or in use
    static constexpr int K = 0, Q = K + 2 * K_BYTES, COLS = Q + STAGES * Q_BYTES;
    static constexpr int RED = COLS + CSTAGES * static_cast<int>(sizeof(Columns));   // f32 [4][2 KEYS]
    static constexpr int BAR = RED + 4 * 2 * KEYS * 4;
    enum { KFULL, KEMPTY, QFULL, QEMPTY = QFULL + STAGES, CFULL = QEMPTY + STAGES, CEMPTY = CFULL + CSTAGES,
           SFULL = CEMPTY + CSTAGES, SEMPTY = SFULL + 2, DRAIN = SEMPTY + 2, NBAR };
    static constexpr int TMEM_AT = BAR + NBAR * 8, BYTES = TMEM_AT + 16 + 1024;
    static_assert(BYTES <= 227 * 1024 && Q % 1024 == 0 && COLS % 16 == 0 && BAR % 8 == 0, "shared memory");
};
constexpr int MANY_THREADS = 768;   // products, row operands, columns and an idle warp; widening; 4 x 4 of sums

constexpr int TURN_ROWS = 8;
__device__ __forceinline__ long long first_row(const AttendArgs& g, int start, int b)
{
    return (static_cast<long long>(start) * g.group / TURN_ROWS + min(b, start)) * TURN_ROWS;
}
// The coefficients of a kv head.
template <typename C>
__device__ __forceinline__ float* coefficients(const WeighArgs& w, int head)
{
    return reinterpret_cast<float*>(w.operands + w.a.c.kv_heads * w.operand_rows * (C::PARTS * C::KB * 128)) + head * w.operand_rows;
}

// A CTA a row.  It needs none of the attention's results, but what was written before the attention (q, start) is
// visible to the CTAs that wait themselves, not to those that one of them waits for.  (With one that
// waited, the others beside the attention's last CTAs, a prompt of 3314 tokens took 1.5 % less.)
template <int D, typename T>
__global__ void __launch_bounds__(256, 8) kv_weigh_rows_kernel(const WeighArgs w)
{
    using C = Many<D, T>;
    const AttendArgs& g = w.a;
    const int lane = threadIdx.x % 32, r = blockIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    const int b = kv_sequence_of(g.c.start, g.c.batch, r, lane);
    const int first = g.c.start[b], last = g.c.start[b + 1];
    if (r < first || r >= last || first < 0 || last > g.ntok)
        return;
    for (int h = threadIdx.x / 32; h < g.heads; h += 8) {
        const int row = (r - first) * g.group + h % g.group;
        const long long at = first_row(g, first, b) + row;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (lane < D / 4)
            x = load4(static_cast<const T*>(g.q.data) + r * g.q.tok + h * g.q.head + 4 * lane, g.wide);
        // a row that is not finite has no weights
        const bool finite = fabsf(x.x) <= FLT_MAX && fabsf(x.y) <= FLT_MAX && fabsf(x.z) <= FLT_MAX && fabsf(x.w) <= FLT_MAX;
        if (!__all_sync(0xffffffffu, finite))
            x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const size_t block = w.operand_rows * 128;
        const float coef = put_row<D, T>(g, x, w.operands + h / g.group * (C::PARTS * C::KB) * block + at * 128, block, row,
                                         C::KB * block, lane);
        if (lane == 0)
            coefficients<C>(w, h / g.group)[at] = coef;
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(MANY_THREADS, 1) kv_weigh_many_kernel(const WeighArgs w)
{
    using C = Many<D, T>;
    constexpr int GROUP = 2 * KEYS;
    const AttendArgs& g = w.a;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t sbase = raw + pad;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    auto bar = [&](int i) -> uint32_t { return sbase + C::BAR + 8u * static_cast<uint32_t>(i); };
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::TMEM_AT);

    grid_dep_wait();
    // early keys are seen by the most rows: their CTAs come first
    const int units = g.c.batch * g.c.kv_heads, part = blockIdx.x / units;
    Unit u;
    const int unit = blockIdx.x % units;
    if (!unit_of(w, unit / g.c.kv_heads, unit % g.c.kv_heads, u))
        return;
    const int groups = (u.length + GROUP - 1) / GROUP;
    if (part >= groups)
        return;
    if (threadIdx.x == 0) {
        mbar_init(bar(C::KFULL), 4);
        mbar_init(bar(C::KEMPTY), 1);
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(bar(C::QFULL + i), 1);
            mbar_init(bar(C::QEMPTY + i), 1);
        }
        for (int i = 0; i < C::CSTAGES; ++i) {
            mbar_init(bar(C::CFULL + i), 1);
            mbar_init(bar(C::CEMPTY + i), 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(C::SFULL + i), 1);
            mbar_init(bar(C::SEMPTY + i), 8);
        }
        mbar_init(bar(C::DRAIN), 1);
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_at), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;

    // the row tiles [lo, hi) that see keys of a group
    auto range = [&](int group, int& lo, int& hi) {
        const int k0 = group * GROUP;
        lo = hi = 0;
        if (!any_seen(g, u.plo, u.phi, k0, GROUP))
            return;
        lo = static_cast<int>(static_cast<long long>(max(k0 - u.pos0, 0)) * g.group / MOST_ROWS);
        long long end = u.rows;
        if (g.window > 0 && k0 >= g.sinks)
            end = min(end, max(static_cast<long long>(k0) + GROUP - 1 + g.window - u.pos0, 0ll) * g.group);
        hi = static_cast<int>((end + MOST_ROWS - 1) / MOST_ROWS);
    };
    bool ok = true;
    int step = 0, visit = 0;    // steps, and groups with any, so far
    if (warp == 0) {
        const uint32_t lead = elect_one();
        for (int group = part; ok && group < groups; group += w.parts) {
            int lo, hi;
            range(group, lo, hi);
            if (lo >= hi)
                continue;
            ok = warp_wait(w, bar(C::KFULL), visit & 1);
            for (int tile = lo; ok && tile < hi; ++tile, ++step) {
                const int stage = step % C::STAGES;
                const int n = min(MOST_ROWS, u.rows - tile * MOST_ROWS);
                const uint32_t idesc = idesc_f16_f32(KEYS, (n + 15) / 16 * 16);
                ok = warp_wait(w, bar(C::QFULL + stage), step / C::STAGES & 1) &&
                     warp_wait(w, bar(C::SEMPTY + step % 2), (step / 2 & 1) ^ 1);
                if (!ok)
                    break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    product<D, C::PARTS>(lead, tmem + (2 * (step % 2) + k) * MOST_ROWS, sbase + C::K + k * C::K_BYTES,
                                         sbase + C::Q + stage * C::Q_BYTES, C::BLOCK, idesc);
                umma_commit_by(lead, bar(C::SFULL + step % 2));
                umma_commit_by(lead, bar(C::QEMPTY + stage));
            }
            if (ok)
                umma_commit_by(lead, bar(C::KEMPTY));
            ++visit;
        }
        umma_commit_by(lead, bar(C::DRAIN));
        if (lead)
            mbar_drain_wait(bar(C::DRAIN), 0, WAIT_LIMIT_NS, g.wc.err);
        __syncwarp();
    } else if (warp == 1) {
        const size_t block = w.operand_rows * 128;
        const uint8_t* operands = w.operands + u.head * (C::PARTS * C::KB) * block + first_row(g, u.first, u.b) * 128;
        for (int group = part; ok && group < groups; group += w.parts) {
            int lo, hi;
            range(group, lo, hi);
            for (int tile = lo; tile < hi; ++tile, ++step) {
                const int stage = step % C::STAGES;
                ok = warp_wait(w, bar(C::QEMPTY + stage), (step / C::STAGES & 1) ^ 1);
                if (!ok)
                    break;
                if (lane == 0) {
                    const uint8_t* src = operands + static_cast<long long>(tile) * C::BLOCK;
                    mbar_arrive_expect_tx(bar(C::QFULL + stage), C::Q_BYTES);
#pragma unroll
                    for (int i = 0; i < C::PARTS * C::KB; ++i)
                        bulk_g2s(sbase + C::Q + stage * C::Q_BYTES + i * C::BLOCK, src + i * block, C::BLOCK, bar(C::QFULL + stage));
                }
            }
        }
        if (lane == 0) {   // the last fill of each stage lands before the CTA ends
            for (int i = max(0, step - C::STAGES); i < step; ++i)
                mbar_drain_wait(bar(C::QFULL + i % C::STAGES), i / C::STAGES & 1, WAIT_LIMIT_NS, g.wc.err);
        }
        __syncwarp();
    } else if (warp == 2) {
        // four rows a lane, on their way while the place is not free
        const float* coefs = coefficients<C>(w, u.head) + first_row(g, u.first, u.b);
        for (int group = part; ok && group < groups; group += w.parts) {
            int lo, hi;
            range(group, lo, hi);
            for (int tile = lo; tile < hi; ++tile, ++step) {
                const int cstage = step % C::CSTAGES;
                const float4 coef = *reinterpret_cast<const float4*>(coefs + static_cast<long long>(tile) * MOST_ROWS + 4 * lane);
                float f[4] = {coef.x, coef.y, coef.z, coef.w};
                float2 stats[4];
                int pos[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = tile * MOST_ROWS + 4 * lane + i, token = row / g.group;
                    const bool there = row < u.rows;
                    pos[i] = there ? u.pos0 + token : -1;
                    stats[i] = there ? g.stats[(u.first + token) * static_cast<size_t>(g.heads) + u.head * g.group + row % g.group]
                                     : make_float2(0.0f, 0.0f);
                    f[i] = stats[i].y > 0.0f ? f[i] : 0.0f;   // none: 2^0, times 0
                }
                ok = warp_wait(w, bar(C::CEMPTY + cstage), (step / C::CSTAGES & 1) ^ 1);
                if (!ok)
                    break;
                Columns* cols = reinterpret_cast<Columns*>(smem + C::COLS) + cstage;
                *reinterpret_cast<float4*>(cols->coef + 4 * lane) = make_float4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<float4*>(cols->minus + 4 * lane) = make_float4(-stats[0].x, -stats[1].x, -stats[2].x, -stats[3].x);
                *reinterpret_cast<float4*>(cols->inv + 4 * lane) = make_float4(stats[0].y, stats[1].y, stats[2].y, stats[3].y);
                *reinterpret_cast<int4*>(cols->pos + 4 * lane) = make_int4(pos[0], pos[1], pos[2], pos[3]);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(C::CFULL + cstage));
            }
        }
    } else if (warp >= 4 && warp < 8) {
        const int t = threadIdx.x - 128;
        for (int group = part; ok && group < groups; group += w.parts) {
            int lo, hi;
            range(group, lo, hi);
            if (lo >= hi)
                continue;
            KeyCodes<D> codes[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = (group * GROUP + k * KEYS + t) / KV_PAGE;
                const int page = i * KV_PAGE < u.length ? u.table[i] : -1;
                const bool there = page >= 0 && page < g.c.num_pages;
                codes[k].get(g.c.pages + (static_cast<size_t>(there ? page : 0) * g.c.kv_heads + u.head) * Piece<D>::BYTES,
                             t % KV_PAGE, there);
            }
            ok = warp_wait(w, bar(C::KEMPTY), (visit & 1) ^ 1);
            if (!ok)
                break;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                codes[k].widen(smem + C::K + k * C::K_BYTES, t);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(C::KFULL));
            ++visit;
        }
    } else if (warp >= 8) {
        // Of every other step a warpgroup takes half of the rows, with both halves of the keys: what it reads of
        // a row then serves two keys of a thread.
        const int s = warp / 4 - 2, part_of = s / 2, odd = s % 2, t = threadIdx.x % KEYS;
        const uint32_t s_at = tmem + 2 * odd * MOST_ROWS + (static_cast<uint32_t>(t & ~31) << 16);
        float* red = reinterpret_cast<float*>(smem + C::RED);   // [4][GROUP]
        for (int group = part; group < groups; group += w.parts) {
            int lo, hi;
            range(group, lo, hi);
            const int k0 = group * GROUP;
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            for (int tile = lo; ok && tile < hi; ++tile, ++step) {
                if (step % 2 != odd)
                    continue;
                const int cstage = step % C::CSTAGES;
                const Columns* cols = reinterpret_cast<const Columns*>(smem + C::COLS) + cstage;
                const int row0 = tile * MOST_ROWS, n = min(MOST_ROWS, u.rows - row0);
                const int c0 = part_of * (MOST_ROWS / 2), c1 = min(n, c0 + MOST_ROWS / 2);
                ok = warp_wait(w, bar(C::CFULL + cstage), step / C::CSTAGES & 1) && warp_wait(w, bar(C::SFULL + odd), step / 2 & 1);
                if (!ok)
                    break;
                tc_fence_after();
                const bool plain = n % 16 == 0 && all_seen(g, u.pos0 + row0 / g.group, u.pos0 + (row0 + n - 1) / g.group, k0, GROUP);
                for (int c = c0; c < c1; c += 16) {
                    float x[2][16];
                    tmem_ld16x2_wait(s_at + c, s_at + MOST_ROWS + c, x[0], x[1]);
                    const Constants<16> at(cols, c);
                    if (plain)
                        add_columns<false>(g, x, at, cols, c, c1, k0 + t, sum);
                    else
                        add_columns<true>(g, x, at, cols, c, c1, k0 + t, sum);
                }
                release(bar(C::SEMPTY + odd), lane);
                if (lane == 0)
                    mbar_arrive(bar(C::CEMPTY + cstage));
            }
            // the four warpgroups' sums, two of them a half of the keys each
            red[s * GROUP + t] = sum[0].x + sum[0].y;
            red[s * GROUP + KEYS + t] = sum[1].x + sum[1].y;
            ok = named_bar_and(2, 512, ok);
            if (!ok)
                break;
            const int j = s * KEYS + t, key = k0 + j;
            if (s < 2 && key < u.length) {
                const int page = u.table[key / KV_PAGE];
                if (page >= 0 && page < g.c.num_pages) {
                    const size_t at = (static_cast<size_t>(page) * g.c.kv_heads + u.head) * KV_PAGE + key % KV_PAGE;
                    const float got = (red[j] + red[GROUP + j]) + (red[2 * GROUP + j] + red[3 * GROUP + j]);
                    w.out[at] = (key < u.pos0 ? w.decay * w.in[at] : 0.0f) + got;
                } else {
                    *g.c.bad = 1u;
                }
            }
            if (group + w.parts < groups)
                named_bar_sync(2, 512);   // what the next group overwrites is read
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ from scores
// The attention for few rows has left its scores, so that K is not read again: 4 bytes a row and key
// for the 72 of a key.  Half a warp has a page, a lane four keys: 9 us for a token on 131071 keys, 32
// heads on 8 (16.8 MB of scores and 8.4 of weights, from L2 for the most part; a warp a page, two keys a
// lane, took 16), 22 us for 64 sequences of up to 8192 (50 MB).  Pages past the ones there was room for
// (a max_kv that is too low) are computed here, value by value.
constexpr int FINISH_WARPS = 4, FINISH_PAGES = 2 * FINISH_WARPS;   // of a CTA at once

template <typename T>
__device__ __forceinline__ const T* query_of(const AttendArgs& g, const Unit& u, int row)
{
    return static_cast<const T*>(g.q.data) + (u.first + row / g.group) * g.q.tok + (u.head * g.group + row % g.group) * g.q.head;
}
// The attention's 2^-e of a row, by which the row is in units of its coefficient: q . k itself may pass f32.
template <int D, typename T>
__device__ __noinline__ float row_scale(const WeighArgs& w, const Unit& u, int row)
{
    const T* q = query_of<T>(w.a, u, row);
    float a = 0.0f;
#pragma unroll 1
    for (int d = 0; d < D; ++d)
        a = fmaxf(a, fabsf(Elt<T>::to(q[d])));
    return kv_pow2(-kv_exponent(a));
}
template <int D, typename T>
__device__ __noinline__ float4 scores_again(const WeighArgs& w, const Unit& u, const uint8_t* piece, int row, float scale, int slot)
{
    const T* q = query_of<T>(w.a, u, row);
    float x[4];
#pragma unroll 1
    for (int h = 0; h < 4; ++h) {
        x[h] = 0.0f;
#pragma unroll 1
        for (int gr = 0; gr < D / 32; ++gr) {
            const uint32_t* code = reinterpret_cast<const uint32_t*>(piece + Piece<D>::k_chunk(slot + h, gr));
            const float s = __half2float(*reinterpret_cast<const __half*>(piece + Piece<D>::k_scale(slot + h, gr)));
#pragma unroll 1
            for (int i = 0; i < 32; ++i) {
                const int n = code[i / 8] >> (4 * (i / 2 % 4) + 16 * (i % 2)) & 15;
                x[h] = fmaf(Elt<T>::to(q[32 * gr + i]) * scale, s * static_cast<float>(n - 8), x[h]);
            }
        }
    }
    return make_float4(x[0], x[1], x[2], x[3]);
}

template <int D, typename T>
__global__ void __launch_bounds__(FINISH_WARPS * 32, 10) kv_finish_weights_kernel(const WeighArgs w)
{
    const AttendArgs& g = w.a;
    __shared__ float4 rows[MOST_ROWS];   // coefficient, reference, 1 / sum; 2^-e where scores are computed here
    grid_dep_wait();
    const int part = blockIdx.x % w.parts, unit = blockIdx.x / w.parts;
    Unit u;
    if (!unit_of(w, unit / g.c.kv_heads, unit % g.c.kv_heads, u))
        return;
    const int n = min(u.rows, g.score_rows), pages = (u.length + KV_PAGE - 1) / KV_PAGE;
    if (part * FINISH_PAGES >= pages)
        return;
    for (int r = threadIdx.x; r < n; r += FINISH_WARPS * 32) {
        const float2 stats = g.stats[(u.first + r / g.group) * static_cast<size_t>(g.heads) + u.head * g.group + r % g.group];
        // a row that is no number adds nothing
        rows[r] = make_float4(g.coef[static_cast<size_t>(unit) * g.score_rows + r], stats.x, stats.y,
                              pages > g.score_pages ? row_scale<D, T>(w, u, r) : 0.0f);
    }
    __syncthreads();
    const bool still = w.in == w.out && w.decay == 1.0f;
    const int slot = threadIdx.x % 16 * 4;
    for (int i = part * FINISH_PAGES + threadIdx.x / 16; i < pages; i += w.parts * FINISH_PAGES) {
        const int kbase = i * KV_PAGE, key = kbase + slot;
        const int page = u.table[i];
        if (page < 0 || page >= g.c.num_pages) {
            *g.c.bad = 1u;
            continue;
        }
        const bool used = any_seen(g, u.plo, u.phi, kbase, KV_PAGE);
        if (!used && still && kbase + KV_PAGE <= u.pos0)
            continue;   // nothing changes
        const size_t piece = static_cast<size_t>(page) * g.c.kv_heads + u.head, at = piece * KV_PAGE + slot;
        const float4 old = key < u.pos0 ? *reinterpret_cast<const float4*>(w.in + at) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (used) {
            const float* scores = g.scores + (static_cast<size_t>(unit) * g.score_pages + i) * g.score_rows * KV_PAGE + slot;
            auto add = [&](float4 x, float4 c) {
                if (c.z > 0.0f) {
                    sum.x = fmaf(kv_ex2(fmaf(x.x, c.x, -c.y)), c.z, sum.x);
                    sum.y = fmaf(kv_ex2(fmaf(x.y, c.x, -c.y)), c.z, sum.y);
                    sum.z = fmaf(kv_ex2(fmaf(x.z, c.x, -c.y)), c.z, sum.z);
                    sum.w = fmaf(kv_ex2(fmaf(x.w, c.x, -c.y)), c.z, sum.w);
                }
            };
            for (int r0 = 0; r0 < n; r0 += w.tile_rows) {
                // a tile of the attention has looked at the pages that one of its rows sees
                const int r1 = min(r0 + w.tile_rows, n);
                const int plo = u.pos0 + r0 / g.group, phi = u.pos0 + (r1 - 1) / g.group;
                if (kbase > phi || (g.window > 0 && i < max(plo - g.window + 1, 0) / KV_PAGE && kbase >= g.sinks))
                    continue;
                if (i < g.score_pages) {
                    for (int r = r0; r < r1; r += 4) {
                        float4 x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            x[k] = *reinterpret_cast<const float4*>(scores + min(r + k, r1 - 1) * KV_PAGE);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (r + k < r1)
                                add(x[k], rows[r + k]);
                    }
                    continue;
                }
                for (int r = r0; r < r1; ++r) {
                    float4 x = scores_again<D, T>(w, u, g.c.pages + piece * Piece<D>::BYTES, r, rows[r].w, slot);
                    const uint64_t m = kv_seen_bits(u.pos0 + r / g.group, kbase, g.window, g.sinks) >> slot;
                    x.x = m & 1u ? x.x : -INFINITY;
                    x.y = m & 2u ? x.y : -INFINITY;
                    x.z = m & 4u ? x.z : -INFINITY;
                    x.w = m & 8u ? x.w : -INFINITY;
                    add(x, rows[r]);
                }
            }
        }
        const float4 got = make_float4((key < u.pos0 ? w.decay * old.x : 0.0f) + sum.x,
                                       (key + 1 < u.pos0 ? w.decay * old.y : 0.0f) + sum.y,
                                       (key + 2 < u.pos0 ? w.decay * old.z : 0.0f) + sum.z,
                                       (key + 3 < u.pos0 ? w.decay * old.w : 0.0f) + sum.w);
        if (key + 3 < u.length) {
            *reinterpret_cast<float4*>(w.out + at) = got;
        } else {
            if (key < u.length)
                w.out[at] = got.x;
            if (key + 1 < u.length)
                w.out[at + 1] = got.y;
            if (key + 2 < u.length)
                w.out[at + 2] = got.z;
        }
    }
}

template <int D, typename T>
cudaError_t launch_finish(WeighArgs a, long long keys, cudaStream_t s)
{
    const long long units = static_cast<long long>(a.a.c.batch) * a.a.c.kv_heads, pages = (keys + KV_PAGE - 1) / KV_PAGE;
    // the chip's 10 CTAs an SM, or 4 pages a half warp where lengths are uneven
    const long long whole = (pages + FINISH_PAGES - 1) / FINISH_PAGES;
    long long parts = 10 * 152 / units > whole / 4 ? 10 * 152 / units : whole / 4;
    parts = parts < whole ? parts : whole;
    parts = parts < 0x7fffffffll / units ? parts : 0x7fffffffll / units;
    a.parts = static_cast<int>(parts < 1 ? 1 : parts);
    count_launch();
    return launch_dependent(kv_finish_weights_kernel<D, T>, dim3(static_cast<unsigned int>(units * a.parts)),
                            dim3(FINISH_WARPS * 32), s, a);
}

template <int D, typename T>
cudaError_t launch_weigh(WeighArgs a, long long keys, cudaStream_t s)
{
    const long long units = static_cast<long long>(a.a.c.batch) * a.a.c.kv_heads;
    auto parts = [&](long long pieces, long long want) {
        want = want < pieces ? want : pieces;
        want = want < 0x7fffffffll / units ? want : 0x7fffffffll / units;
        return static_cast<int>(want < 1 ? 1 : want);
    };
    if (a.operand_rows == 0) {
        static std::atomic<uint64_t> done{0};
        cudaError_t e = kv_allow_smem(kv_weigh_few_kernel<D, T>, 226 * 1024, &done);
        if (e != cudaSuccess)
            return e;
        const FewLayout l = Few<D, T>::layout(a.cols);
        count_launch();
        return launch_dependent_smem(kv_weigh_few_kernel<D, T>, dim3(152), dim3(FEW_THREADS), static_cast<size_t>(l.bytes), s, a, l);
    }
    using C = Many<D, T>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = kv_allow_smem(kv_weigh_many_kernel<D, T>, C::BYTES, &done);
    if (e != cudaSuccess)
        return e;
    count_launch();
    if ((e = launch_dependent(kv_weigh_rows_kernel<D, T>, dim3(static_cast<unsigned int>(a.a.ntok)), dim3(256), s, a)) !=
        cudaSuccess)
        return e;
    const long long groups = (keys + 2 * KEYS - 1) / (2 * KEYS);
    a.parts = parts(groups, groups);
    count_launch();
    return launch_dependent_smem(kv_weigh_many_kernel<D, T>, dim3(static_cast<unsigned int>(units * a.parts)),
                                 dim3(MANY_THREADS), C::BYTES, s, a);
}

}  // namespace

size_t weigh_bytes(int dtype, int heads, int kv_heads, int dim, int batch, int ntok, int max_q, int* cols,
                   long long* operand_rows)
{
    const long long group = heads / kv_heads, rows = (max_q < ntok ? max_q : ntok) * group;
    *cols = static_cast<int>(rows < 16 ? 16 : rows > MOST_ROWS ? MOST_ROWS : (rows + 15) / 16 * 16);
    // up to 7 rows between two sequences, and the last step's copies past the last row
    *operand_rows = rows <= MOST_ROWS ? 0
                                      : (static_cast<long long>(ntok) * group / TURN_ROWS + (batch < ntok ? batch : ntok)) * TURN_ROWS +
                                            MOST_ROWS;
    const size_t row = static_cast<size_t>(dtype == KV_F32 ? 2 : 1) * dim * 2 + 4;
    return static_cast<size_t>(*operand_rows) * kv_heads * row;
}

cudaError_t launch_kv_weigh(const WeighArgs& a, int dim, int dtype, int max_kv, cudaStream_t s)
{
    const long long room = static_cast<long long>(a.a.c.max_pages) * KV_PAGE, keys = max_kv < room ? max_kv : room;
    if (dim == 128)
        return dtype == KV_F32   ? launch_weigh<128, float>(a, keys, s)
               : dtype == KV_F16 ? launch_weigh<128, __half>(a, keys, s)
                                 : launch_weigh<128, __nv_bfloat16>(a, keys, s);
    return dtype == KV_F32   ? launch_weigh<64, float>(a, keys, s)
           : dtype == KV_F16 ? launch_weigh<64, __half>(a, keys, s)
                             : launch_weigh<64, __nv_bfloat16>(a, keys, s);
}

cudaError_t launch_kv_finish_weights(const WeighArgs& a, int dim, int dtype, int max_kv, cudaStream_t s)
{
    const long long room = static_cast<long long>(a.a.c.max_pages) * KV_PAGE, keys = max_kv < room ? max_kv : room;
    if (dim == 128)
        return dtype == KV_F32   ? launch_finish<128, float>(a, keys, s)
               : dtype == KV_F16 ? launch_finish<128, __half>(a, keys, s)
                                 : launch_finish<128, __nv_bfloat16>(a, keys, s);
    return dtype == KV_F32   ? launch_finish<64, float>(a, keys, s)
           : dtype == KV_F16 ? launch_finish<64, __half>(a, keys, s)
                             : launch_finish<64, __nv_bfloat16>(a, keys, s);
}

}  // namespace mmq
