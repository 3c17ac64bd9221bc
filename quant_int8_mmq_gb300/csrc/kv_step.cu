// kv_step.cu -- attention over the 4-bit cache for few rows per sequence: single tokens
// and a few drafted ones.
//
//   o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m),   x_j = scale log2(e) q . k_j,  visible j
//
// The cache is read once and its bytes bound the work: a 128-value head costs 144 bytes a
// key.  What has to keep up with them is the widening of the codes, so the layout is made
// for registers: a lane's 16-byte load is exactly its part of an operand of mma m16n8k16,
// and widening a pair of codes takes one logic operation, a quarter of a shift and one or
// two f16x2 operations that also apply the scale.
//   S = Q K^T   Q is the 16-row operand, 8 keys the columns; lane (n, t) supplies a quarter
//               t of key n's values.
//   O^T = V^T P^T   V is the 16-row operand (lane (n, t): two of its D/8 values by two pairs
//               of keys), and the accumulators of S are, in place, the operand P^T.
// Transposed, O needs D/4 accumulators a lane for 8 rows whether P has one or two parts;
// as P V they were twice that, and 12 warps an SM instead of 16.
//
// A row is a query token and one of the heads that share the kv head.  Tiles:
//   f32 rows: 8, the operand's 16 rows holding the f16 parts of q = 2^e (hi + lo), and
//     P = hi + lo as two products into the same accumulators: 22 bits at each operand;
//   16-bit rows: 8 in the same way with P rounded to f16, or, where there are more, 16
//     (q has no low part worth having: 2^-e q is exact in f16 down to 2^-24).
//
// A CTA is 4 warps; each takes every fourth of the CTA's pages through its own ring of
// bulk copies, with its own running reference and sums, and the four are joined in shared
// memory.  When there are few tiles, or sequences of uneven length, the visible pages are
// cut into parts.  A part goes to a cluster of up to 8 CTAs, which share its pages evenly
// whatever their number turns out to be and join their sums through distributed shared
// memory; only what takes more parts than one goes by the workspace and a second kernel.
//
// The tensor cores cut sums toward zero at every product, 8 a page for f32 rows.  Those set
// their sums aside every RUN pages of a warp and go on from zero: what is left is the cut of
// 128 products, 6e-6 of values of one sign whatever the length (one sum over 20000 keys lost
// 3.2e-5, over 131072 keys 2.2e-4).  A part is that long a warp only where a cluster takes up
// to 128 pages a CTA or where max_kv is far too low; the others pay for the test (one token on
// 131071 keys, 47.8 us for 46.0).
//
// What bounds it: chains of dependent instructions, some 1500 a page for widening and products,
// at the 4 warps a scheduler that the registers hold: an instruction issues in 57 % of the
// cycles, and no pipe is over 45 % busy.  On GB300: one token on 131071 keys, 32 f32 heads of
// 128 on 8, 48 us (3.2 TB/s), on 524288 keys 158 us (3.8 TB/s); 64 sequences of 95 to 8192
// keys, bf16, 92 us (3.4 TB/s).  A copy reaches 6.8 TB/s.
//
// The 16-row tiles of 128 values spill: 20 of a page's instructions are loads and stores of
// spilled registers (1.3 %); the other builds have 3 or none.
#include <atomic>

#include "kv.cuh"

namespace mmq {
namespace {

constexpr int WARPS = 4;
constexpr int STAGES = 2;   // half pieces (K or V) a warp's ring holds
constexpr int RUN = 16;     // pages that a warp's accumulators sum up before f32 rows set them aside

// Row tiles (see above).
enum Mode { HI_LO = 0, ONE_PART = 1, WIDE = 2 };

template <int D, int MODE>
struct StepSmem {
    static constexpr int ROWS = MODE == WIDE ? 16 : 8;
    static constexpr int HALF = Piece<D>::V_CODES;                  // bytes of a piece's K or V
    static constexpr int RING = 0;                                  // [WARPS][STAGES] halves
    static constexpr int Q = RING + WARPS * STAGES * HALF;
    static constexpr int COEF = Q + 16 * D * 2;                     // f32 per row
    static constexpr int ML = COEF + ROWS * 4;                      // float2 [WARPS][ROWS]
    static constexpr int BAR = ML + WARPS * ROWS * 8;
    static constexpr int BYTES = BAR + WARPS * STAGES * 8;
    static constexpr int OROW = D + 4;                              // f32 of a joined row, in the idle ring
    static_assert(WARPS * ROWS * OROW * 4 <= Q, "joined sums fit the ring");
    static_assert(Q % 16 == 0 && ML % 8 == 0 && BAR % 8 == 0, "alignment");
};

__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// WEIGH: the scores of the keys, if there is room for them, and the rows' statistics are left for
// kv_weigh.cu: 48.5 us for 47.2 on 131071 keys, 32 heads on 8, f32.
template <int D, typename T, int MODE, bool WEIGH>
__global__ void __launch_bounds__(WARPS * 32, MODE == WIDE ? 3 : D == 128 ? 4 : 6) kv_step_kernel(const AttendArgs g)
{
    using P = Piece<D>;
    using S = StepSmem<D, MODE>;
    constexpr int ROWS = S::ROWS, SETS = ROWS / 8;   // rows n and, of a wide tile, n + 8
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int n = lane / 4, t = lane % 4;

    grid_dep_wait();
    // the unit: a part of the pages for one row tile of one sequence's kv head
    int id = blockIdx.x / g.cluster;
    const int rank = blockIdx.x % g.cluster;
    if (id == static_cast<int>(gridDim.x) / g.cluster - 1) {
        if (rank == 0)
            kv_clear_others<D, T, WEIGH>(g, static_cast<long long>(g.row_tiles) * ROWS);
        return;
    }
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
    const int nrow = min(ROWS, rows_b - row0);
    const int pos0 = max(g.c.length[b], 0) - rows_b / g.group;
    const int room = g.c.max_pages * KV_PAGE;
    // positions of the tile's first and last row; keys [0, kend) are looked at
    const int plo = pos0 + row0 / g.group, phi = pos0 + (row0 + nrow - 1) / g.group;
    const int kend = min(max(phi + 1, 0), room);
    if (threadIdx.x == 0 && phi + 1 > room)
        *g.c.bad = 1u;
    // pages: the sinks' that lie wholly before the window's first, then the window's
    const int klo = g.window > 0 ? min(max(plo - g.window + 1, 0), kend) : 0;
    const int page_lo = klo / KV_PAGE;
    const int nsink = min((min(g.sinks, kend) + KV_PAGE - 1) / KV_PAGE, page_lo);
    const int npage = nsink + (kend + KV_PAGE - 1) / KV_PAGE - page_lo;
    // the last part takes what the caller's max_kv did not foresee
    const long long part0 = static_cast<long long>(split) * g.part_pages;
    const int part1 = split == g.nsplit - 1 ? npage : static_cast<int>(min(part0 + g.part_pages, static_cast<long long>(npage)));
    const int flat_rows = g.ntok * g.heads;
    if (g.nsplit > 1 && part0 >= npage) {   // nothing here: say so and leave
        if (rank == 0 && threadIdx.x < nrow) {
            const int row = row0 + threadIdx.x;
            g.part_ml[static_cast<size_t>(split) * flat_rows + static_cast<size_t>(first + row / g.group) * g.heads +
                      head * g.group + row % g.group] = make_float2(-INFINITY, 0.0f);
        }
        return;
    }
    // this CTA's share: a page a warp at least
    const int share = max((part1 - static_cast<int>(part0) + g.cluster - 1) / g.cluster, WARPS);
    const int i0 = static_cast<int>(part0) + rank * share + warp;
    const int i_end = min(static_cast<int>(part0) + (rank + 1) * share, part1);
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
    // verification only: the first CTA's first page is left out (never armed, never copied), so
    // that the wait for it runs out
    constexpr int WITHHELD = 0x7fffffff;
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
                } else if (g.wc.withhold_fill >= 0 && blockIdx.x == 0 && warp == 0 && k + lane == 0) {
                    ids = WITHHELD;
                }
            }
        }
        const int pid = __shfl_sync(0xffffffffu, ids, k % 32);
        if (pid >= 0) {
            flying |= 1u << fill;
            if (lane == 0 && pid != WITHHELD) {
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
        const int e = kv_exponent(a);
        const float f = kv_pow2(-e);
        if (lane < D / 4) {
            uint2 hi, lo;
            kv_split2(x.x * f, x.y * f, hi.x, lo.x);
            kv_split2(x.z * f, x.w * f, hi.y, lo.y);
            // as the operand's lanes read it: values D/4 t .. of row n (and n + 8), four a step
            const int step = 4 * lane % (D / 4) / 4, owner = r % 8 * 4 + 4 * lane / (D / 4);
            uint32_t* at = reinterpret_cast<uint32_t*>(smem + S::Q + (step * 32 + owner) * 16);
            if constexpr (MODE == WIDE) {
                at[r / 8] = hi.x;
                at[2 + r / 8] = hi.y;
            } else {
                *reinterpret_cast<uint4*>(at) = make_uint4(hi.x, lo.x, hi.y, lo.y);
            }
        }
        if (lane == 0) {
            const float coef = fminf(fmaxf(g.scale_log2 * kv_pow2(e), 1e-38f), 1e38f);
            *reinterpret_cast<float*>(smem + S::COEF + 4 * r) = coef;
            if (WEIGH && r < nrow && row0 + r < g.score_rows)   // every part's CTAs write the same
                g.coef[(static_cast<size_t>(b) * g.c.kv_heads + head) * g.score_rows + row0 + r] = coef;
        }
    }
    __syncthreads();

    // the operand Q, read again for every two octets of keys: kept in registers (32 of them) it
    // left the rest too few to run ahead (524288 keys, 32 heads on 8: 158 us for 154, before f32 rows
    // set sums aside)
    const uint4* qf = reinterpret_cast<const uint4*>(smem + S::Q) + lane;   // step j at 32 j
    float coef[SETS], ref[SETS], sum[SETS];
    int pos[SETS];   // the row sees keys up to here, -1: no row
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
        coef[i] = *reinterpret_cast<const float*>(smem + S::COEF + 4 * (n + 8 * i));
        pos[i] = n + 8 * i < nrow ? pos0 + (row0 + n + 8 * i) / g.group : -1;
        ref[i] = -INFINITY;
        sum[i] = 0.0f;
    }
    // values D/8 n + 2 j (elements 0, 1) and D/8 n + 2 j + 1 (2, 3) of rows 2t, 2t + 1 (and + 8)
    float o[SETS][D / 16][4];
#pragma unroll
    for (int i = 0; i < SETS; ++i)
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
            o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.0f;

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
    // Long parts of f32 rows (see above): sums set aside, in local memory, so that the loop's
    // registers are not needed for them.  `ahead` tells the pages so far.
    [[maybe_unused]] volatile float aside[D / 4 + 1];
    auto any_aside = [&] { return MODE == HI_LO && ahead > 2 * RUN + STAGES - 1; };
    auto set_aside = [&] {
        const bool any = any_aside();
#pragma unroll
        for (int j = 0; j < D / 4; ++j) {
            aside[j] = any ? aside[j] + o[0][j / 4][j % 4] : o[0][j / 4][j % 4];
            o[0][j / 4][j % 4] = 0.0f;
        }
        aside[D / 4] = any ? aside[D / 4] + sum[0] : sum[0];
        sum[0] = 0.0f;
    };
    for (int i = i0; i < i_end; i += WARPS) {
        if constexpr (MODE == HI_LO) {
            if (ahead % (2 * RUN) == STAGES - 1 && ahead > 2 * RUN)
                set_aside();
        }
        const uint8_t* page = next_half();
        if (page == nullptr) {
            if (!ok)
                break;
            next_half();   // its other half is not there either
            continue;
        }
        const int kbase = (i < nsink ? i : page_lo + i - nsink) * KV_PAGE;

        // x[o]: keys 8o + 2t and 8o + 2t + 1 of row n (and n + 8); two octets of keys at a time
        float x[8][SETS][2];
#pragma unroll
        for (int oct = 0; oct < 8; oct += 2) {
            uint32_t w[2][D / 32];
            __half2 s[2], sb[2];
            // f32 rows: two sums a key, as the tensor cores cut sums toward zero at every step
            constexpr int SUMS = MODE == HI_LO ? 2 : 1;
            float c[2][SUMS][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int token = 8 * (oct + h) + n;
                if constexpr (D == 128) {
                    const uint4 v = *reinterpret_cast<const uint4*>(page + P::k_chunk(token, t));
                    w[h][0] = v.x, w[h][1] = v.y, w[h][2] = v.z, w[h][3] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(page + P::k_chunk(token, t / 2) + t % 2 * 8);
                    w[h][0] = v.x, w[h][1] = v.y;
                }
                s[h] = __half2half2(*reinterpret_cast<const __half*>(page + P::k_scale(token, D == 128 ? t : t / 2)));
                sb[h] = kv_addend(s[h]);
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const uint4 q = qf[32 * j];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t v = w[h][j / 2];
                    const uint32_t b0 = kv_h2u(j % 2 ? kv_widen<2>(v, s[h], sb[h]) : kv_widen<0>(v, s[h], sb[h]));
                    const uint32_t b1 = kv_h2u(j % 2 ? kv_widen<3>(v, s[h], sb[h]) : kv_widen<1>(v, s[h], sb[h]));
                    if (j < SUMS)
                        mma16816_first(c[h][j % SUMS], q.x, q.y, q.z, q.w, b0, b1);
                    else
                        mma16816(c[h][j % SUMS], q.x, q.y, q.z, q.w, b0, b1);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if constexpr (MODE == WIDE) {
                        x[oct + h][0][e] = c[h][0][e];
                        x[oct + h][1][e] = c[h][0][e + 2];
                    } else if constexpr (MODE == HI_LO) {
                        x[oct + h][0][e] = (c[h][0][e + 2] + c[h][1][e + 2]) + (c[h][0][e] + c[h][1][e]);
                    } else {
                        x[oct + h][0][e] = c[h][0][e] + c[h][0][e + 2];
                    }
                }
        }

        // keys past the row's own, before its window (and not among the sinks)
        const bool whole = kbase + KV_PAGE - 1 <= plo &&
                           (g.window == 0 || kbase > phi - g.window || kbase + KV_PAGE <= g.sinks);
        if (!whole) {
#pragma unroll
            for (int i = 0; i < SETS; ++i) {
                const uint64_t m = kv_seen_bits(pos[i], kbase, g.window, g.sinks) >> (2 * t);
#pragma unroll
                for (int oct = 0; oct < 8; ++oct)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if ((m >> (8 * oct + e) & 1u) == 0)
                            x[oct][i][e] = -INFINITY;
            }
        }

        if constexpr (WEIGH) {
            const int at = kbase / KV_PAGE;
            if (at < g.score_pages) {
                float* to = g.scores +
                            ((static_cast<size_t>(b) * g.c.kv_heads + head) * g.score_pages + at) * g.score_rows * KV_PAGE + 2 * t;
#pragma unroll
                for (int i = 0; i < SETS; ++i) {
                    const int row = n + 8 * i;
                    if (row < nrow && row0 + row < g.score_rows) {
#pragma unroll
                        for (int oct = 0; oct < 8; ++oct)
                            *reinterpret_cast<float2*>(to + (row0 + row) * KV_PAGE + 8 * oct) =
                                make_float2(x[oct][i][0], x[oct][i][1]);
                    }
                }
            }
        }

        float base[SETS];
        bool raise = false;
        float next[SETS];
#pragma unroll
        for (int i = 0; i < SETS; ++i) {
            float top = x[0][i][0];
#pragma unroll
            for (int oct = 0; oct < 8; ++oct)
                top = fmaxf(top, fmaxf(x[oct][i][0], x[oct][i][1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)) * coef[i];
            const bool up = top > ref[i] + KV_REF_LIMIT;   // also the first visible key: ref is -inf until then
            next[i] = up ? top - kv_ref_below<T>() : ref[i];
            raise |= up;
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int i = 0; i < SETS; ++i) {
                const float f = next[i] == ref[i] ? 1.0f : kv_ex2(ref[i] - next[i]);
                ref[i] = next[i];
                sum[i] *= f;
                const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    o[i][j][0] *= f0;
                    o[i][j][1] *= f1;
                    o[i][j][2] *= f0;
                    o[i][j][3] *= f1;
                }
                if constexpr (MODE == HI_LO) {
                    if (any_aside()) {
#pragma unroll
                        for (int j = 0; j < D / 4; ++j)
                            aside[j] = aside[j] * (j % 2 ? f1 : f0);
                        aside[D / 4] = aside[D / 4] * f;
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < SETS; ++i)
            base[i] = ref[i] == -INFINITY ? 0.0f : ref[i];

        page = next_half();
        if (!ok)
            break;
        page -= P::V_CODES;
        const int held = min(kend - kbase, KV_PAGE);
        float page_sum = 0.0f;   // f32 rows: a page's weights together do not vanish beside a large sum
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {   // keys 16 kk .. 16 kk + 15
            uint32_t hi[SETS][2], lo[2];
#pragma unroll
            for (int i = 0; i < SETS; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float p0 = kv_ex2(fmaf(x[2 * kk + h][i][0], coef[i], -base[i]));
                    const float p1 = kv_ex2(fmaf(x[2 * kk + h][i][1], coef[i], -base[i]));
                    (MODE == HI_LO ? page_sum : sum[i]) += p0 + p1;
                    if constexpr (MODE == HI_LO)
                        kv_split2(p0, p1, hi[i][h], lo[h]);
                    else
                        hi[i][h] = kv_h2u(__floats2half2_rn(p0, p1));
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
            auto step = [&](float (&c0)[4], float (&c1)[4], const uint32_t (&a)[4], const uint32_t (&b)[4], uint32_t p0,
                            uint32_t p1) {
                mma16816(c0, a[0], a[1], a[2], a[3], p0, p1);
                mma16816(c1, b[0], b[1], b[2], b[3], p0, p1);
            };
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {   // values 4 j .. 4 j + 3 of the lane's
                const uint32_t a[4] = {kv_h2u(kv_widen<0>(w[0][j], s[0], sb[0])), kv_h2u(kv_widen<1>(w[0][j], s[0], sb[0])),
                                       kv_h2u(kv_widen<0>(w[1][j], s[1], sb[1])), kv_h2u(kv_widen<1>(w[1][j], s[1], sb[1]))};
                const uint32_t b[4] = {kv_h2u(kv_widen<2>(w[0][j], s[0], sb[0])), kv_h2u(kv_widen<3>(w[0][j], s[0], sb[0])),
                                       kv_h2u(kv_widen<2>(w[1][j], s[1], sb[1])), kv_h2u(kv_widen<3>(w[1][j], s[1], sb[1]))};
#pragma unroll
                for (int i = 0; i < SETS; ++i)
                    step(o[i][2 * j], o[i][2 * j + 1], a, b, hi[i][0], hi[i][1]);
                if constexpr (MODE == HI_LO)
                    step(o[0][2 * j], o[0][2 * j + 1], a, b, lo[0], lo[1]);
            }
        }
        if constexpr (MODE == HI_LO)
            sum[0] += page_sum;
    }
    if (any_aside()) {
#pragma unroll
        for (int j = 0; j < D / 4; ++j)
            o[0][j / 4][j % 4] += aside[j];
        sum[0] += aside[D / 4];
    }
    if (!ok) {   // a wait ran out: the copies in flight still have to land before the CTA ends
        const bool withheld = __shfl_sync(0xffffffffu, ids, 0) == WITHHELD;   // both halves of it, nothing else
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
            if (flying >> s & 1u && !withheld)
                mbar_drain_wait(bar + 8 * s, parity >> s & 1u, WAIT_LIMIT_NS, g.wc.err);
    }

    grid_dep_launch();
    // join the warps
    __syncthreads();
    float2* ml = reinterpret_cast<float2*>(smem + S::ML);
    float* os = reinterpret_cast<float*>(smem + S::RING);
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        if (t == 0)
            ml[warp * ROWS + n + 8 * i] = make_float2(ref[i], sum[i]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
                *reinterpret_cast<float4*>(os + (warp * ROWS + 2 * t + e + 8 * i) * S::OROW + n * (D / 8) + 4 * j) =
                    make_float4(o[i][2 * j][e], o[i][2 * j][e + 2], o[i][2 * j + 1][e], o[i][2 * j + 1][e + 2]);
    }
    __syncthreads();

    constexpr int LANES = WARPS * 32 / ROWS;   // threads a row
    constexpr int GROUPS = D / (4 * LANES);    // of four values a thread
    const int r = threadIdx.x / LANES, l = threadIdx.x % LANES;
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
    float4 v[GROUPS];
    auto add = [](float4& a, float k, float4 b) {
        a.x += k * b.x;
        a.y += k * b.y;
        a.z += k * b.z;
        a.w += k * b.w;
    };
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
        v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            add(v[j], f[w], *reinterpret_cast<const float4*>(os + (w * ROWS + r) * S::OROW + 4 * (LANES * j + l)));
    }
    if (g.cluster > 1) {
        __syncthreads();   // everyone has read the warps' sums, the CTA's go over them
        if (l == 0)
            ml[r] = make_float2(top, total);
#pragma unroll
        for (int j = 0; j < GROUPS; ++j)
            *reinterpret_cast<float4*>(os + r * S::OROW + 4 * (LANES * j + l)) = v[j];
        cluster_sync();
        if (rank == 0) {
            const uint32_t ml_at = smem_u32(ml + r), os_at = smem_u32(os + r * S::OROW + 4 * l);
            float all = top;
            for (int c = 1; c < g.cluster; ++c)
                all = fmaxf(all, ld_cluster_f32(cluster_map(ml_at, c)));
            const float own = top == -INFINITY ? 0.0f : kv_ex2(top - all);
            total *= own;
#pragma unroll
            for (int j = 0; j < GROUPS; ++j)
                v[j] = make_float4(own * v[j].x, own * v[j].y, own * v[j].z, own * v[j].w);
            for (int c = 1; c < g.cluster; ++c) {
                const float ref_c = ld_cluster_f32(cluster_map(ml_at, c));
                const float k = ref_c == -INFINITY ? 0.0f : kv_ex2(ref_c - all);
                total += k * ld_cluster_f32(cluster_map(ml_at + 4, c));
#pragma unroll
                for (int j = 0; j < GROUPS; ++j)
                    add(v[j], k, ld_cluster_f32x4(cluster_map(os_at + 16 * LANES * j, c)));
            }
            top = all;
        }
        cluster_sync();    // the first CTA has read the others' sums
        if (rank != 0)
            return;
    }
    if (r >= nrow)
        return;
    const int row = row0 + r;
    const long long token = first + row / g.group;
    const int h = head * g.group + row % g.group;
    const size_t at = static_cast<size_t>(split) * flat_rows + static_cast<size_t>(token) * g.heads + h;
    if (g.nsplit > 1 && l == 0)
        g.part_ml[at] = make_float2(top, total);
    if (WEIGH && g.nsplit == 1 && l == 0)
        g.stats[at] = kv_row_stats(top, total);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;   // a row that sees no key is zero
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
        const int d = 4 * (LANES * j + l);
        if (g.nsplit > 1)
            *reinterpret_cast<float4*>(g.part + at * D + d) = v[j];
        else
            store4(static_cast<T*>(g.out.data) + token * g.out.tok + h * g.out.head + d,
                   make_float4(v[j].x * inv, v[j].y * inv, v[j].z * inv, v[j].w * inv), g.wide);
    }
}

// Joins the nsplit sums of each row: a CTA per row, its warps taking the splits in turn.
constexpr int JOIN_WARPS = 4;
template <int D, typename T, bool WEIGH>
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
    if (WEIGH && threadIdx.x == 0)
        g.stats[flat] = kv_row_stats(top, total);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    store4(static_cast<T*>(g.out.data) + static_cast<long long>(flat / g.heads) * g.out.tok +
               static_cast<long long>(flat % g.heads) * g.out.head + d,
           v, g.wide);
}

template <int D, typename T, int MODE, bool WEIGH>
cudaError_t launch_step(const AttendArgs& a, cudaStream_t s)
{
    constexpr int BYTES = StepSmem<D, MODE>::BYTES;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = kv_allow_smem(kv_step_kernel<D, T, MODE, WEIGH>, BYTES, &done);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned int>(a.cluster);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned int>(
        a.cluster * (static_cast<long long>(a.nsplit) * a.c.kv_heads * a.row_tiles * a.c.batch + 1)));
    cfg.blockDim = dim3(WARPS * 32);
    cfg.dynamicSmemBytes = BYTES;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, kv_step_kernel<D, T, MODE, WEIGH>, a);
}
template <int D, typename T, int MODE>
cudaError_t launch_step(const AttendArgs& a, cudaStream_t s)
{
    return a.stats ? launch_step<D, T, MODE, true>(a, s) : launch_step<D, T, MODE, false>(a, s);
}

template <int D>
cudaError_t launch_step(const AttendArgs& a, int dtype, cudaStream_t s)
{
    if (dtype == KV_F32)
        return launch_step<D, float, HI_LO>(a, s);
    if (a.tile_rows == 8)
        return dtype == KV_F16 ? launch_step<D, __half, ONE_PART>(a, s) : launch_step<D, __nv_bfloat16, ONE_PART>(a, s);
    return dtype == KV_F16 ? launch_step<D, __half, WIDE>(a, s) : launch_step<D, __nv_bfloat16, WIDE>(a, s);
}

template <int D, typename T>
cudaError_t launch_join(const AttendArgs& a, cudaStream_t s)
{
    count_launch();
    return launch_dependent(a.stats ? kv_join_kernel<D, T, true> : kv_join_kernel<D, T, false>, dim3(static_cast<unsigned int>(a.ntok) * a.heads),
                            dim3(JOIN_WARPS * 32), s, a);
}

}  // namespace

cudaError_t launch_kv_step(const AttendArgs& a, int dim, int dtype, cudaStream_t s)
{
    return dim == 128 ? launch_step<128>(a, dtype, s) : launch_step<64>(a, dtype, s);
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
