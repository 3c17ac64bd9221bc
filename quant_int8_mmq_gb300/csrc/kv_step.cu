// kv_step.cu -- attention over the 4-bit cache for few rows per sequence: single tokens
// and a few drafted ones.
//
//   o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m),   x_j = scale log2(e) q . k_j,  visible j
//
// The cache is read once and its bytes bound the work: a 128-value head costs 144 bytes a
// key.  What has to keep up with them is the widening of the codes, so the layout is made
// for registers: a lane's 16-byte load is exactly its part of the tensor-core operand
// (mma m16n8k16: keys are the 8 columns of Q K^T, each lane supplying a quarter of its
// key's values; 16 keys are the depth of P V, each lane supplying two pairs of keys for
// D/8 values), and widening a pair of codes takes a mask, mostly a shift, and one fma
// that also applies the scale.
//
// A tile is 8 rows (a row is a query token and one of the heads that share the kv head).
// They fill the 16 operand rows as 8 high parts and 8 low parts of f16 each, q = 2^e
// (hi + lo) and p = hi + lo with 22 bits, while the cached values are exact in f16, so
// the products carry f32 precision at the price of the 16-bit instruction.
//
// A CTA is 4 warps; each takes every fourth of the CTA's pages through its own ring of
// bulk copies, with its own running reference and sums, and the four are joined in shared
// memory.  When there are few tiles the visible pages are split over nsplit CTAs, whose
// sums go to the workspace and are joined by a second kernel.
#include <atomic>

#include "kv.cuh"

namespace mmq {
namespace {

constexpr int WARPS = 4;
constexpr int STAGES = 3;   // half pieces (K or V) a warp's ring holds
constexpr int ROWS = KV_STEP_ROWS;

template <int D>
struct StepSmem {
    static constexpr int QROW = D * 2 + 16;                         // padded row of f16
    static constexpr int HALF = Piece<D>::V_CODES;                  // bytes of a piece's K or V
    static constexpr int RING = 0;                                  // [WARPS][STAGES] halves
    static constexpr int Q = RING + WARPS * STAGES * HALF;
    static constexpr int COEF = Q + 2 * ROWS * QROW;                // f32 per row
    static constexpr int ML = COEF + ROWS * 4;                      // float2 [WARPS][ROWS]
    static constexpr int BAR = ML + WARPS * ROWS * 8;
    static constexpr int BYTES = BAR + WARPS * STAGES * 8;
    static constexpr int OROW = D + 4;                              // f32 of a joined row, in the idle ring
    static_assert(WARPS * ROWS * OROW * 4 <= Q, "joined sums fit the ring");
    static_assert(Q % 16 == 0 && ML % 8 == 0 && BAR % 8 == 0, "alignment");
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D, typename T>
__global__ void __launch_bounds__(WARPS * 32, D == 128 ? 3 : 4) kv_step_kernel(const AttendArgs g)
{
    using P = Piece<D>;
    using S = StepSmem<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int n = lane / 4, t = lane % 4;

    grid_dep_wait();
    // the unit: a split of the pages for one row tile of one sequence's kv head
    int id = blockIdx.x;
    const int split = id % g.nsplit;
    id /= g.nsplit;
    const int head = id % g.c.kv_heads;
    id /= g.c.kv_heads;
    const int tile = id % g.row_tiles, b = id / g.row_tiles;
    const int first = g.c.start[b], last = g.c.start[b + 1];
    if (first < 0 || last <= first || last > g.ntok)
        return;
    const int rows_b = (last - first) * g.group, row0 = tile * ROWS;
    if (row0 >= rows_b)
        return;
    if (threadIdx.x == 0 && tile == 0 && (rows_b + ROWS - 1) / ROWS > g.row_tiles)
        *g.c.bad = 1u;   // more new tokens than the caller's max_q: rows past it are not computed
    const int nrow = min(ROWS, rows_b - row0);
    const long long pos0 = static_cast<long long>(g.c.length[b]) - rows_b / g.group;
    const long long room = static_cast<long long>(g.c.max_pages) * KV_PAGE;
    // positions of the tile's first and last row; keys [0, kend) are looked at
    const long long plo = pos0 + row0 / g.group, phi = pos0 + (row0 + nrow - 1) / g.group;
    const int kend = static_cast<int>(min(max(phi + 1, 0ll), room));
    if (threadIdx.x == 0 && phi + 1 > room)
        *g.c.bad = 1u;
    // pages: the sinks' that lie wholly before the window's first, then the window's
    const int klo = g.window > 0 ? static_cast<int>(min(max(plo - g.window + 1, 0ll), static_cast<long long>(kend))) : 0;
    const int page_lo = klo / KV_PAGE;
    const int nsink = min((min(g.sinks, kend) + KV_PAGE - 1) / KV_PAGE, page_lo);
    const int npage = nsink + (kend + KV_PAGE - 1) / KV_PAGE - page_lo;
    // the last part takes what the caller's max_kv did not foresee
    const long long part0 = static_cast<long long>(split) * g.part_pages;
    const int i_end = split == g.nsplit - 1 ? npage : static_cast<int>(min(part0 + g.part_pages, static_cast<long long>(npage)));
    const int flat_rows = g.ntok * g.heads;
    if (g.nsplit > 1 && part0 >= npage) {   // nothing here: say so and leave
        if (threadIdx.x < nrow) {
            const int row = row0 + threadIdx.x;
            g.part_ml[static_cast<size_t>(split) * flat_rows + static_cast<size_t>(first + row / g.group) * g.heads +
                      head * g.group + row % g.group] = make_float2(-INFINITY, 0.0f);
        }
        return;
    }

    const int i0 = static_cast<int>(part0) + warp;
    const uint32_t sbase = smem_u32(smem);
    const uint32_t ring = sbase + S::RING + warp * STAGES * S::HALF;
    const uint32_t bar = sbase + S::BAR + warp * STAGES * 8;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i)
            mbar_init(bar + 8 * i, 1);
        fence_barrier_init();
    }
    __syncwarp();

    // the warp's pages are i0, i0 + WARPS, ...; ids of 32 of them at a time, one per lane
    const int* table = g.c.table + static_cast<size_t>(b) * g.c.max_pages;
    int ids = -1, ahead = 0;   // halves asked for so far: K, V of the first page, K, ...
    int fill = 0;              // their next stage
    uint32_t flying = 0;       // bit s: stage s holds or awaits a half
    auto fetch = [&] {
        const int k = ahead / 2;
        if (ahead % 64 == 0) {
            const int j = i0 + (k + lane) * WARPS;
            ids = -1;
            if (j < i_end) {
                ids = table[j < nsink ? j : page_lo + j - nsink];
                if (ids < 0 || ids >= g.c.num_pages) {
                    *g.c.bad = 1u;
                    ids = -1;
                }
            }
        }
        const int pid = __shfl_sync(0xffffffffu, ids, k % 32);
        if (pid >= 0) {
            flying |= 1u << fill;
            if (lane == 0) {
                fence_proxy_async_smem();   // the stage's last half was read with ordinary loads
                mbar_arrive_expect_tx(bar + 8 * fill, S::HALF);
                bulk_g2s(ring + fill * S::HALF,
                         g.c.pages + (static_cast<size_t>(pid) * g.c.kv_heads + head) * P::BYTES + ahead % 2 * S::HALF,
                         S::HALF, bar + 8 * fill);
            }
        }
        ++ahead;
        fill = fill + 1 == STAGES ? 0 : fill + 1;
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
        fetch();

    // query rows: 2^-e q as hi and lo f16, coefficient 2^e scale log2(e)
    for (int r = warp; r < ROWS; r += WARPS) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < nrow && lane < D / 4) {
            const int row = row0 + r;
            const T* q = static_cast<const T*>(g.q.data) + (first + row / g.group) * g.q.tok +
                         (head * g.group + row % g.group) * g.q.head;
            x = load4(q + 4 * lane, g.wide);
        }
        float a = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
        const int e = a > 0.0f && a < INFINITY ? ilogbf(a) : 0;
        if (lane < D / 4) {
            uint2 hi, lo;
            kv_split2(scalbnf(x.x, -e), scalbnf(x.y, -e), hi.x, lo.x);
            kv_split2(scalbnf(x.z, -e), scalbnf(x.w, -e), hi.y, lo.y);
            *reinterpret_cast<uint2*>(smem + S::Q + r * S::QROW + lane * 8) = hi;
            *reinterpret_cast<uint2*>(smem + S::Q + (ROWS + r) * S::QROW + lane * 8) = lo;
        }
        if (lane == 0)
            *reinterpret_cast<float*>(smem + S::COEF + 4 * r) = scalbnf(g.scale_log2, e);
    }
    __syncthreads();

    // operand rows n (hi) and n + 8 (lo): lane t holds values D/4 t .. D/4 t + D/4 - 1
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        const uint2 hi = *reinterpret_cast<const uint2*>(smem + S::Q + n * S::QROW + (D / 4 * t + 4 * j) * 2);
        const uint2 lo = *reinterpret_cast<const uint2*>(smem + S::Q + (ROWS + n) * S::QROW + (D / 4 * t + 4 * j) * 2);
        qf[j][0] = hi.x;
        qf[j][1] = lo.x;
        qf[j][2] = hi.y;
        qf[j][3] = lo.y;
    }
    const float coef = *reinterpret_cast<const float*>(smem + S::COEF + 4 * n);
    const long long pos = n < nrow ? pos0 + (row0 + n) / g.group : -1;   // row n sees keys up to here
    const long long low = g.window > 0 ? pos - g.window + 1 : 0;         // and from here, or below g.sinks

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
        o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float ref = -INFINITY, sum = 0.0f;

    uint32_t parity = 0;   // bit s: parity of stage s's next arrival
    int take = 0;          // stage of the next half
    bool ok = true;
    // the next half, once it is there: its bytes, or null for a page that is not in the pool
    auto next_half = [&]() -> const uint8_t* {
        __syncwarp();
        fetch();
        const int stage = take;
        take = take + 1 == STAGES ? 0 : take + 1;
        if ((flying >> stage & 1u) == 0)
            return nullptr;
        ok = __all_sync(0xffffffffu, mbar_wait(bar + 8 * stage, parity >> stage & 1u, g.wc.limit_ns, g.wc.err));
        if (!ok)
            return nullptr;
        parity ^= 1u << stage;
        flying &= ~(1u << stage);
        return smem + S::RING + (warp * STAGES + stage) * S::HALF;
    };
    for (int i = i0; i < i_end; i += WARPS) {
        const uint8_t* page = next_half();
        if (page == nullptr) {
            if (!ok)
                break;
            next_half();   // its other half is not there either
            continue;
        }
        const long long kbase = static_cast<long long>(i < nsink ? i : page_lo + i - nsink) * KV_PAGE;

        // x[o]: keys 8o + 2t and 8o + 2t + 1 of row n
        float x[8][2];
#pragma unroll
        for (int oct = 0; oct < 8; ++oct) {
            const int token = 8 * oct + n;
            uint32_t w[D / 32];
            if constexpr (D == 128) {
                const uint4 v = *reinterpret_cast<const uint4*>(page + P::k_chunk(token, t));
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(page + P::k_chunk(token, t / 2) + t % 2 * 8);
                w[0] = v.x, w[1] = v.y;
            }
            const __half2 s = __half2half2(
                *reinterpret_cast<const __half*>(page + P::k_scale(token, D == 128 ? t : t / 2)));
            const __half2 sb = kv_addend(s);
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                mma16816(c, qf[2 * j][0], qf[2 * j][1], qf[2 * j][2], qf[2 * j][3], kv_h2u(kv_widen<0>(w[j], s, sb)),
                         kv_h2u(kv_widen<1>(w[j], s, sb)));
                mma16816(c, qf[2 * j + 1][0], qf[2 * j + 1][1], qf[2 * j + 1][2], qf[2 * j + 1][3],
                         kv_h2u(kv_widen<2>(w[j], s, sb)), kv_h2u(kv_widen<3>(w[j], s, sb)));
            }
            x[oct][0] = (c[0] + c[2]) * coef;
            x[oct][1] = (c[1] + c[3]) * coef;
        }

        // keys past the row's own, before its window (and not among the sinks)
        const bool whole = kbase + KV_PAGE - 1 <= plo &&
                           (g.window == 0 || kbase > phi - g.window || kbase + KV_PAGE <= g.sinks);
        if (!whole) {
            const int to = static_cast<int>(min(max(pos - kbase, -1ll), static_cast<long long>(KV_PAGE)));
            const int from = static_cast<int>(min(max(low - kbase, 0ll), static_cast<long long>(KV_PAGE)));
            const int sink = static_cast<int>(min(max(g.sinks - kbase, 0ll), static_cast<long long>(KV_PAGE)));
#pragma unroll
            for (int oct = 0; oct < 8; ++oct)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = 8 * oct + 2 * t + e;
                    if (j > to || (j < from && j >= sink))
                        x[oct][e] = -INFINITY;
                }
        }

        float top = x[0][0];
#pragma unroll
        for (int oct = 0; oct < 8; ++oct)
            top = fmaxf(top, fmaxf(x[oct][0], x[oct][1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const bool raise = top > ref + KV_REF_LIMIT;   // also the first visible key: ref is -inf until then
        if (__any_sync(0xffffffffu, raise)) {
            const float next = raise ? top - KV_REF_BELOW : ref;
            const float f = raise ? kv_ex2(ref - next) : 1.0f;
            ref = next;
            sum *= f;
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[j][e] *= f;
        }
        const float base = ref == -INFINITY ? 0.0f : ref;

        page = next_half();
        if (!ok)
            break;
        page -= P::V_CODES;
        const int held = static_cast<int>(min(kend - kbase, static_cast<long long>(KV_PAGE)));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {   // keys 16 kk .. 16 kk + 15
            uint32_t a[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float p0 = kv_ex2(x[2 * kk + h][0] - base), p1 = kv_ex2(x[2 * kk + h][1] - base);
                sum += p0 + p1;
                kv_split2(p0, p1, a[2 * h], a[2 * h + 1]);
            }
            uint32_t w[2][D / 32];
            __half2 s[2], sb[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int pair = 8 * kk + 4 * h + t;
                if constexpr (D == 128) {
                    const uint4 v = *reinterpret_cast<const uint4*>(page + P::v_chunk(pair, n));
                    w[h][0] = v.x, w[h][1] = v.y, w[h][2] = v.z, w[h][3] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(page + P::v_chunk(pair, n / 2) + n % 2 * 8);
                    w[h][0] = v.x, w[h][1] = v.y;
                }
                uint32_t sc = *reinterpret_cast<const uint32_t*>(page + P::v_scale(pair, n * (D / 8) / KV_GROUP));
                // slots without a token hold anything, and 0 times a scale that is no number is none
                if (held < KV_PAGE)
                    sc = 2 * pair + 1 < held ? sc : 2 * pair < held ? sc & 0xffffu : 0u;
                s[h] = kv_u2h(sc);
                sb[h] = kv_addend(s[h]);
            }
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                mma16816(o[4 * j], a[0], a[1], a[2], a[3], kv_h2u(kv_widen<0>(w[0][j], s[0], sb[0])),
                         kv_h2u(kv_widen<0>(w[1][j], s[1], sb[1])));
                mma16816(o[4 * j + 1], a[0], a[1], a[2], a[3], kv_h2u(kv_widen<1>(w[0][j], s[0], sb[0])),
                         kv_h2u(kv_widen<1>(w[1][j], s[1], sb[1])));
                mma16816(o[4 * j + 2], a[0], a[1], a[2], a[3], kv_h2u(kv_widen<2>(w[0][j], s[0], sb[0])),
                         kv_h2u(kv_widen<2>(w[1][j], s[1], sb[1])));
                mma16816(o[4 * j + 3], a[0], a[1], a[2], a[3], kv_h2u(kv_widen<3>(w[0][j], s[0], sb[0])),
                         kv_h2u(kv_widen<3>(w[1][j], s[1], sb[1])));
            }
        }
    }
    if (!ok) {   // a wait ran out: the copies in flight still have to land before the CTA ends
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
            if (flying >> s & 1u)
                mbar_drain_wait(bar + 8 * s, parity >> s & 1u, WAIT_LIMIT_NS, g.wc.err);
    }

    // join the warps: column c of the output operand holds values D/8 c .. D/8 c + D/8 - 1
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    __syncthreads();
    float2* ml = reinterpret_cast<float2*>(smem + S::ML);
    if (t == 0)
        ml[warp * ROWS + n] = make_float2(ref, sum);
    float* os = reinterpret_cast<float*>(smem + S::RING);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            float4 v;
            v.x = o[4 * j][c] + o[4 * j][c + 2];
            v.y = o[4 * j + 1][c] + o[4 * j + 1][c + 2];
            v.z = o[4 * j + 2][c] + o[4 * j + 2][c + 2];
            v.w = o[4 * j + 3][c] + o[4 * j + 3][c + 2];
            *reinterpret_cast<float4*>(os + (warp * ROWS + n) * S::OROW + (2 * t + c) * (D / 8) + 4 * j) = v;
        }
    __syncthreads();

    const int r = threadIdx.x / 16, l = threadIdx.x % 16;   // 16 threads a row
    if (r >= nrow)
        return;
    float top = -INFINITY, total = 0.0f, f[WARPS];
#pragma unroll
    for (int w = 0; w < WARPS; ++w)
        top = fmaxf(top, ml[w * ROWS + r].x);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const float2 v = ml[w * ROWS + r];
        f[w] = v.x == -INFINITY ? 0.0f : kv_ex2(v.x - top);
        total += f[w] * v.y;
    }
    const int row = row0 + r;
    const long long token = first + row / g.group;
    const int h = head * g.group + row % g.group;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        const int d = 64 * j + 4 * l;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float4 p = *reinterpret_cast<const float4*>(os + (w * ROWS + r) * S::OROW + d);
            v.x += f[w] * p.x;
            v.y += f[w] * p.y;
            v.z += f[w] * p.z;
            v.w += f[w] * p.w;
        }
        const size_t flat = static_cast<size_t>(token) * g.heads + h;
        if (g.nsplit == 1) {
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;   // a row that sees no key is zero
            v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            store4(static_cast<T*>(g.out.data) + token * g.out.tok + h * g.out.head + d, v, g.wide);
        } else {
            const size_t at = static_cast<size_t>(split) * flat_rows + flat;
            *reinterpret_cast<float4*>(g.part + at * D + d) = v;
            if (l == 0 && j == 0)
                g.part_ml[at] = make_float2(top, total);
        }
    }
}

// Joins the nsplit sums of each row: a CTA per row, its warps taking the splits in turn.
constexpr int JOIN_WARPS = 4;
template <int D, typename T>
__global__ void __launch_bounds__(JOIN_WARPS * 32) kv_join_kernel(const AttendArgs g)
{
    __shared__ float4 part[JOIN_WARPS][32];
    __shared__ float psum[JOIN_WARPS];
    constexpr int L = D / 4;          // lanes of one row
    constexpr int SETS = 32 / L;      // splits that a warp takes at once
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int set = lane / L, d = lane % L * 4;
    const size_t flat = blockIdx.x, rows = static_cast<size_t>(g.ntok) * g.heads;
    grid_dep_wait();

    float top = -INFINITY;
    for (int s = lane; s < g.nsplit; s += 32)
        top = fmaxf(top, g.part_ml[s * rows + flat].x);
#pragma unroll
    for (int k = 1; k < 32; k <<= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));

    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float total = 0.0f;
#pragma unroll 4
    for (int s = warp * SETS + set; s < g.nsplit; s += JOIN_WARPS * SETS) {
        const size_t at = s * rows + flat;
        const float2 ml = g.part_ml[at];
        if (ml.x == -INFINITY && ml.y == 0.0f)
            continue;   // saw no key; its sums may not have been written
        const float4 p = *reinterpret_cast<const float4*>(g.part + at * D + d);
        const float f = kv_ex2(ml.x - top);
        total += f * ml.y;
        v.x += f * p.x;
        v.y += f * p.y;
        v.z += f * p.z;
        v.w += f * p.w;
    }
    part[warp][lane] = v;
    if constexpr (SETS == 2)
        total += __shfl_xor_sync(0xffffffffu, total, L);
    if (lane == 0)
        psum[warp] = total;
    __syncthreads();
    if (threadIdx.x >= L)
        return;
    total = 0.0f;
    v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < JOIN_WARPS; ++w) {
        total += psum[w];
#pragma unroll
        for (int i = 0; i < SETS; ++i) {
            const float4 p = part[w][i * L + threadIdx.x];
            v.x += p.x;
            v.y += p.y;
            v.z += p.z;
            v.w += p.w;
        }
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    store4(static_cast<T*>(g.out.data) + static_cast<long long>(flat / g.heads) * g.out.tok +
               static_cast<long long>(flat % g.heads) * g.out.head + d,
           v, g.wide);
}

template <int D, typename T>
cudaError_t launch_step(const AttendArgs& a, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = kv_allow_smem(kv_step_kernel<D, T>, StepSmem<D>::BYTES, &done);
    if (e != cudaSuccess)
        return e;
    const unsigned int grid = static_cast<unsigned int>(static_cast<long long>(a.nsplit) * a.c.kv_heads * a.row_tiles *
                                                        a.c.batch);
    count_launch();
    return launch_dependent_smem(kv_step_kernel<D, T>, dim3(grid), dim3(WARPS * 32), StepSmem<D>::BYTES, s, a);
}

template <int D, typename T>
cudaError_t launch_join(const AttendArgs& a, cudaStream_t s)
{
    count_launch();
    return launch_dependent(kv_join_kernel<D, T>, dim3(static_cast<unsigned int>(a.ntok) * a.heads),
                            dim3(JOIN_WARPS * 32), s, a);
}

}  // namespace

cudaError_t launch_kv_step(const AttendArgs& a, int dim, int dtype, cudaStream_t s)
{
    if (dim == 128)
        return dtype == KV_F32   ? launch_step<128, float>(a, s)
               : dtype == KV_F16 ? launch_step<128, __half>(a, s)
                                 : launch_step<128, __nv_bfloat16>(a, s);
    return dtype == KV_F32   ? launch_step<64, float>(a, s)
           : dtype == KV_F16 ? launch_step<64, __half>(a, s)
                             : launch_step<64, __nv_bfloat16>(a, s);
}

cudaError_t launch_kv_join(const AttendArgs& a, int dim, int dtype, cudaStream_t s)
{
    if (dim == 128)
        return dtype == KV_F32   ? launch_join<128, float>(a, s)
               : dtype == KV_F16 ? launch_join<128, __half>(a, s)
                                 : launch_join<128, __nv_bfloat16>(a, s);
    return dtype == KV_F32   ? launch_join<64, float>(a, s)
           : dtype == KV_F16 ? launch_join<64, __half>(a, s)
                             : launch_join<64, __nv_bfloat16>(a, s);
}

}  // namespace mmq
