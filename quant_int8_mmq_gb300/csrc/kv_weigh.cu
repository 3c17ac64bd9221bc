// kv_weigh.cu -- the weight that each key of the 4-bit cache receives from the new tokens' rows:
//
//   out[j] = decay in[j] (tokens that were there) + sum over rows 2^(x_j - ref) / sum,
//   x_j = scale log2(e) q . k_j
//
// with each row's reference and sum from the attention that ran before.  S^T = K Q^T on the
// tensor cores: keys are the 128 lanes of tensor memory and rows its columns, so a key's sum
// over the rows stays in one thread's register and nothing is added up across threads or
// CTAs; what a column needs (coefficient, reference, 1 / sum) is read by whole warps at once.
// K is widened to f16, exactly, from the codes; rows are scaled by a power of two and, where
// they are f32, split in two f16 parts.
//
// kv_weigh_few_kernel, up to 128 rows per sequence and kv head: the rows stay in shared memory
// and the keys stream by, 128 a step, their codes through a ring of bulk copies.  One warpgroup
// widens (a thread a key) and issues the products, two take every other step's S each.
//
// kv_weigh_many_kernel: 256 keys stay in shared memory and the rows stream by, 128 a step, as
// operands that kv_weigh_rows_kernel has laid out in the workspace.  Four warpgroups, one for each
// half of the keys and every other step.
#include <type_traits>

#include "kv.cuh"

namespace mmq {
namespace {

constexpr int KEYS = 128;       // lanes of tensor memory
constexpr int MOST_ROWS = 128;  // columns of a step

// What a row's column needs, in shared memory and (many rows) in the workspace.
struct alignas(16) Columns {
    float coef[MOST_ROWS], ref[MOST_ROWS], inv[MOST_ROWS];
    int pos[MOST_ROWS];
};

__device__ __forceinline__ bool wait(const WeighArgs& w, uint32_t bar, uint32_t parity)
{
    return mbar_wait_asleep(bar, parity, w.a.wc.limit_ns, w.a.wc.err);
}
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
__device__ __forceinline__ bool unit_of(const WeighArgs& w, int id, Unit& u)
{
    const AttendArgs& g = w.a;
    u.head = id % g.c.kv_heads;
    u.b = id / g.c.kv_heads;
    u.first = g.c.start[u.b];
    const int last = g.c.start[u.b + 1];
    if (u.first < 0 || last <= u.first || last > g.ntok)
        return false;
    const int new_tokens = last - u.first, counted = min(new_tokens, w.max_q);
    if (new_tokens > counted && threadIdx.x == 0)
        *g.c.bad = 1u;
    u.rows = counted * g.group;
    u.length = min(max(g.c.length[u.b], 0), g.c.max_pages * KV_PAGE);
    u.pos0 = max(g.c.length[u.b], 0) - new_tokens;
    u.plo = u.pos0;
    u.phi = u.pos0 + counted - 1;
    u.table = g.c.table + static_cast<size_t>(u.b) * g.c.max_pages;
    return u.rows > 0;
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
    // row t of [64-value block][128 keys] tiles, 128-byte swizzle
    __device__ __forceinline__ void widen(uint8_t* dst, int t) const
    {
#pragma unroll
        for (int gr = 0; gr < D / 32; ++gr) {
            const uint32_t both = gr < 2 ? scale.x : scale.y;
            const __half2 s = kv_u2h(__byte_perm(both, 0, gr % 2 ? 0x3232 : 0x1010)), sb = kv_addend(s);
            const uint32_t v[4] = {code[gr].x, code[gr].y, code[gr].z, code[gr].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4*>(dst + gr / 2 * KEYS * 128 + t * 128 + ((gr % 2 * 4 + i) ^ (t & 7)) * 16) =
                    make_uint4(kv_h2u(kv_widen<0>(v[i], s, sb)), kv_h2u(kv_widen<1>(v[i], s, sb)),
                               kv_h2u(kv_widen<2>(v[i], s, sb)), kv_h2u(kv_widen<3>(v[i], s, sb)));
        }
    }
};

// One row as operand row r of [64-value block][n rows] tiles, by a warp, an f32 row's low part as
// row r + low; what its column needs.  A row whose statistics are {0, 0} becomes zeros.
template <int D, typename T>
__device__ __forceinline__ void put_row(const AttendArgs& g, const T* q, float2 stats, int pos, uint8_t* dst, int n, int r,
                                        int low, Columns* cols, int lane)
{
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (q && stats.y > 0.0f && lane < D / 4)
        x = load4(q + 4 * lane, g.wide);
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
        uint8_t* at = dst + d / 64 * n * 128 + r * 128 + ((d / 8 % 8 ^ (r & 7)) << 4) + d % 8 * 2;
        *reinterpret_cast<uint2*>(at) = hi;
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<uint2*>(at + low * 128) = lo;   // a multiple of 8 rows: the same turn
    }
    if (lane == 0) {
        cols->coef[r] = fminf(fmaxf(g.scale_log2 * kv_pow2(e), 1e-38f), 1e38f);
        cols->ref[r] = stats.x;
        cols->inv[r] = stats.y;
        cols->pos[r] = pos;
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

// The weights of 16 columns of a key.
template <bool MASKED>
__device__ __forceinline__ void add_columns(const AttendArgs& g, const float (&x)[16], const Columns* cols, int c0, int n,
                                            int key, float2& sum)
{
#pragma unroll
    for (int c = 0; c < 16; c += 4) {
        if (c0 + c >= n)
            break;
        const float4 f = *reinterpret_cast<const float4*>(cols->coef + c0 + c);
        const float4 r = *reinterpret_cast<const float4*>(cols->ref + c0 + c);
        const float4 v = *reinterpret_cast<const float4*>(cols->inv + c0 + c);
        float4 p = make_float4(kv_ex2(fmaf(x[c], f.x, -r.x)), kv_ex2(fmaf(x[c + 1], f.y, -r.y)),
                               kv_ex2(fmaf(x[c + 2], f.z, -r.z)), kv_ex2(fmaf(x[c + 3], f.w, -r.w)));
        if constexpr (MASKED) {
            const int4 pos = *reinterpret_cast<const int4*>(cols->pos + c0 + c);
            auto seen = [&](int i, int at) {
                return c0 + c + i < n && key <= at && (g.window == 0 || key > at - g.window || key < g.sinks);
            };
            p.x = seen(0, pos.x) ? p.x : 0.0f;
            p.y = seen(1, pos.y) ? p.y : 0.0f;
            p.z = seen(2, pos.z) ? p.z : 0.0f;
            p.w = seen(3, pos.w) ? p.w : 0.0f;
        }
        sum = ffma2(make_float2(p.x, p.y), make_float2(v.x, v.y), sum);
        sum = ffma2(make_float2(p.z, p.w), make_float2(v.z, v.w), sum);
    }
}

// ------------------------------------------------------------------ few rows
constexpr int FEW_WARPS = 14;               // widening, two of sums, one that copies, one that issues products
constexpr int COPY_WARP = 12, MMA_WARP = 13;

// f32 rows: the low parts are n more columns, so that K is read once for both.
template <int D, typename T>
struct Few {
    static constexpr int PARTS = sizeof(T) == 4 ? 2 : 1, KB = D / 64;
    static constexpr int K_BYTES = KB * KEYS * 128;
    static constexpr int HALF = Piece<D>::V_CODES;                 // a page's keys
    static constexpr int STAGES = 4, STAGE = 2 * HALF;             // codes on their way
    static constexpr int RING = 2 * K_BYTES, COLS = RING + STAGES * STAGE;
    static constexpr int META = COLS + static_cast<int>(sizeof(Columns));   // int2 [STAGES]: whether its pages are there
    static constexpr int BAR = META + STAGES * 8;
    enum { QFULL, RFULL, REMPTY = RFULL + STAGES, KFULL = REMPTY + STAGES, KEMPTY = KFULL + 2, SFULL = KEMPTY + 2,
           SEMPTY = SFULL + 2, DRAIN = SEMPTY + 2, NBAR };
    static constexpr int TMEM_AT = BAR + NBAR * 8;
    static constexpr int Q = (TMEM_AT + 4 + 1023) / 1024 * 1024;
    static_assert(RING % 16 == 0 && COLS % 16 == 0 && BAR % 8 == 0, "alignment");
    static constexpr int bytes(int n) { return Q + PARTS * KB * n * 128 + 1024; }   // and the alignment
    __host__ __device__ static constexpr int columns(int n)        // of one S in tensor memory
    {
        return n * PARTS <= 32 ? 32 : n * PARTS <= 64 ? 64 : n * PARTS <= 128 ? 128 : 256;
    }
};

template <int D, typename T>
__global__ void __launch_bounds__(FEW_WARPS * 32) kv_weigh_few_kernel(const WeighArgs w)
{
    using C = Few<D, T>;
    using P = Piece<D>;
    const AttendArgs& g = w.a;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t sbase = raw + pad;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    auto bar = [&](int i) -> uint32_t { return sbase + C::BAR + 8u * static_cast<uint32_t>(i); };
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::TMEM_AT);
    Columns* cols = reinterpret_cast<Columns*>(smem + C::COLS);
    int2* meta = reinterpret_cast<int2*>(smem + C::META);

    grid_dep_wait();
    const int part = blockIdx.x % w.parts;
    Unit u;
    if (!unit_of(w, blockIdx.x / w.parts, u))
        return;
    const int n = w.cols, rows = min(u.rows, n);
    if (u.rows > n && threadIdx.x == 0)
        *g.c.bad = 1u;
    const int tiles = (u.length + KEYS - 1) / KEYS;
    if (part >= tiles)
        return;
    const uint32_t columns = C::columns(n);
    if (threadIdx.x == 0) {
        mbar_init(bar(C::QFULL), COPY_WARP);
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(bar(C::RFULL + i), 1);
            mbar_init(bar(C::REMPTY + i), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(C::KFULL + i), 4);
            mbar_init(bar(C::KEMPTY + i), 1);
            mbar_init(bar(C::SFULL + i), 1);
            mbar_init(bar(C::SEMPTY + i), 4);
        }
        mbar_init(bar(C::DRAIN), 1);
        fence_barrier_init();
    }
    if (warp == MMA_WARP) {
        tmem_alloc(smem_u32(tmem_at), 2 * columns);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;

    if (warp < COPY_WARP) {   // the rows, while the first codes are on their way
        for (int r = warp; r < n; r += COPY_WARP) {
            const bool there = r < rows;
            const long long token = u.first + r / g.group;
            const int h = u.head * g.group + r % g.group;
            put_row<D, T>(g, there ? static_cast<const T*>(g.q.data) + token * g.q.tok + h * g.q.head : nullptr,
                          there ? g.stats[token * g.heads + h] : make_float2(0.0f, 0.0f), there ? u.pos0 + r / g.group : -1,
                          smem + C::Q, C::PARTS * n, r, n, cols, lane);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(C::QFULL));
    }

    // the CTA's tiles are part, part + parts, ...; those of which no key is seen are passed over
    auto seen = [&](int tile) { return any_seen(g, u.plo, u.phi, tile * KEYS, KEYS); };
    bool ok = true;
    int step = 0;   // tiles so far of which a key is seen
    if (warp < 4) {
        // ------------------------------------------------------------ widening
        const int t = threadIdx.x;
        for (int tile = part; ok && tile < tiles; tile += w.parts) {
            if (!seen(tile))
                continue;
            const int buf = step % 2, stage = step % C::STAGES;
            ok = warp_wait(w, bar(C::RFULL + stage), step / C::STAGES & 1) &&
                 warp_wait(w, bar(C::KEMPTY + buf), (step / 2 & 1) ^ 1);
            if (!ok)
                break;
            const int2 there = meta[stage];
            KeyCodes<D> codes;
            codes.get(smem + C::RING + stage * C::STAGE + t / KV_PAGE * C::HALF, t % KV_PAGE, t < KV_PAGE ? there.x : there.y);
            codes.widen(smem + buf * C::K_BYTES, t);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(C::KFULL + buf));
                mbar_arrive(bar(C::REMPTY + stage));
            }
            ++step;
        }
    } else if (warp == MMA_WARP) {
        // ------------------------------------------------------------ products
        const uint32_t lead = elect_one(), idesc = idesc_f16_f32(KEYS, C::PARTS * n);
        ok = warp_wait(w, bar(C::QFULL), 0);
        for (int tile = part; ok && tile < tiles; tile += w.parts) {
            if (!seen(tile))
                continue;
            const int buf = step % 2;
            ok = warp_wait(w, bar(C::KFULL + buf), step / 2 & 1) && warp_wait(w, bar(C::SEMPTY + buf), (step / 2 & 1) ^ 1);
            if (!ok)
                break;
            tc_fence_after();
            product<D, 1>(lead, tmem + buf * columns, sbase + buf * C::K_BYTES, sbase + C::Q, C::PARTS * n * 128, idesc);
            umma_commit_by(lead, bar(C::SFULL + buf));
            umma_commit_by(lead, bar(C::KEMPTY + buf));
            ++step;
        }
        umma_commit_by(lead, bar(C::DRAIN));
        if (lead)
            mbar_drain_wait(bar(C::DRAIN), 0, WAIT_LIMIT_NS, g.wc.err);
        __syncwarp();
    } else if (warp == COPY_WARP) {
        // ------------------------------------------------------------ codes: the keys of two pages a step
        // ids of 16 tiles at a time, two lanes each, and those of the next 16 on their way
        auto ids_of = [&](long long k) {
            const long long tile = part + (k + lane / 2) * w.parts, i = 2 * tile + lane % 2;
            return tile < tiles && i * KV_PAGE < u.length ? u.table[i] : -1;
        };
        int ids = -1, later = ids_of(0);
        for (int k = 0, tile = part; tile < tiles; ++k, tile += w.parts) {
            if (k % 16 == 0) {
                ids = later < g.c.num_pages ? later : -1;
                later = ids_of(k + 16);
            }
            if (!seen(tile))
                continue;
            const int p0 = __shfl_sync(0xffffffffu, ids, k % 16 * 2), p1 = __shfl_sync(0xffffffffu, ids, k % 16 * 2 + 1);
            const int stage = step % C::STAGES;
            ok = warp_wait(w, bar(C::REMPTY + stage), (step / C::STAGES & 1) ^ 1);
            if (!ok)
                break;
            if (lane == 0) {
                meta[stage] = make_int2(p0 >= 0, p1 >= 0);
                fence_proxy_async_smem();   // the stage was read with ordinary loads
                mbar_arrive_expect_tx(bar(C::RFULL + stage), ((p0 >= 0) + (p1 >= 0)) * C::HALF);
                const uint32_t dst = sbase + C::RING + stage * C::STAGE;
                const size_t piece = static_cast<size_t>(g.c.kv_heads) * P::BYTES;
                const uint8_t* src = g.c.pages + static_cast<size_t>(u.head) * P::BYTES;
                if (p0 >= 0)
                    bulk_g2s(dst, src + p0 * piece, C::HALF, bar(C::RFULL + stage));
                if (p1 >= 0)
                    bulk_g2s(dst + C::HALF, src + p1 * piece, C::HALF, bar(C::RFULL + stage));
            }
            ++step;
        }
        if (lane == 0)   // the last fill of each stage lands before the CTA ends
            for (int i = max(0, step - C::STAGES); i < step; ++i)
                mbar_drain_wait(bar(C::RFULL + i % C::STAGES), i / C::STAGES & 1, WAIT_LIMIT_NS, g.wc.err);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ sums: a thread a key
        const int buf = warp / 4 - 1, t = threadIdx.x % KEYS;
        const uint32_t s_at = tmem + buf * columns + (static_cast<uint32_t>(t & ~31) << 16);
        int unseen = 0;   // tiles so far of which no key is seen; they go to the warpgroups in turn too
        // the warpgroup's next tile from `tile` on, and whether S has it
        auto next = [&](int tile, bool& used) {
            for (; tile < tiles; tile += w.parts) {
                used = seen(tile);
                if ((used ? step++ : unseen++) % 2 != buf)
                    continue;
                if (used || w.in != w.out || w.decay != 1.0f || tile * KEYS + KEYS > u.pos0)
                    return tile;   // else nothing changes
            }
            return tile;
        };
        auto page_of = [&](int tile) { return tile < tiles && tile * KEYS + t < u.length ? u.table[(tile * KEYS + t) / KV_PAGE] : -1; };
        auto place = [&](int page, int tile) {
            return (static_cast<size_t>(page) * g.c.kv_heads + u.head) * KV_PAGE + (tile * KEYS + t) % KV_PAGE;
        };
        auto had = [&](int page, int tile) {
            return page >= 0 && page < g.c.num_pages && tile * KEYS + t < u.pos0 ? w.in[place(page, tile)] : 0.0f;
        };
        // what the next tile had is on its way while this one's weights are added up, and the page of
        // the one after that
        bool used = false, used1 = false, used2 = false;
        int tile = next(part, used), tile1 = tile < tiles ? next(tile + w.parts, used1) : tile;
        int page = page_of(tile), page1 = page_of(tile1), turn = 0;
        float old = had(page, tile);
        ok = warp_wait(w, bar(C::QFULL), 0);
        while (ok && tile < tiles) {
            const int tile2 = tile1 < tiles ? next(tile1 + w.parts, used2) : tile1, page2 = page_of(tile2);
            const float old1 = had(page1, tile1);
            float2 sum = make_float2(0.0f, 0.0f);
            if (used) {
                ok = warp_wait(w, bar(C::SFULL + buf), turn & 1);
                if (!ok)
                    break;
                ++turn;
                tc_fence_after();
                const bool plain = rows % 4 == 0 && all_seen(g, u.plo, u.phi, tile * KEYS, KEYS);
                for (int c = 0; c < rows; c += 16) {
                    float x[16];
                    if constexpr (C::PARTS == 2) {
                        float lo[16];
                        tmem_ld16x2_wait(s_at + c, s_at + n + c, x, lo);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            x[i] += lo[i];
                    } else {
                        tmem_ld16_wait(s_at + c, x);
                    }
                    if (c + 16 >= rows) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(bar(C::SEMPTY + buf));
                    }
                    if (plain)
                        add_columns<false>(g, x, cols, c, rows, tile * KEYS + t, sum);
                    else
                        add_columns<true>(g, x, cols, c, rows, tile * KEYS + t, sum);
                }
            }
            if (page >= 0 && page < g.c.num_pages)
                w.out[place(page, tile)] = w.decay * old + (sum.x + sum.y);
            else if (tile * KEYS + t < u.length)
                *g.c.bad = 1u;
            tile = tile1;
            page = page1;
            used = used1;
            old = old1;
            tile1 = tile2;
            page1 = page2;
            used1 = used2;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == MMA_WARP)
        tmem_dealloc(tmem, 2 * columns);
}

// ------------------------------------------------------------------ many rows
// Operand tiles in the workspace: 128 rows of one sequence and kv head, [part][64-value block][row],
// and their columns.  Those of sequence b are base(b), base(b) + 1, ...; tiles of a kv head
// lie together.
template <int D, typename T>
struct Many {
    static constexpr int PARTS = sizeof(T) == 4 ? 2 : 1, KB = D / 64;
    static constexpr int BLOCK = MOST_ROWS * 128;
    static constexpr int Q_BYTES = PARTS * KB * BLOCK;
    static constexpr int RECORD = Q_BYTES + static_cast<int>(sizeof(Columns));
    static constexpr int K_BYTES = KB * KEYS * 128;        // of 128 keys
    static constexpr int STAGES = 2, CSTAGES = 4;          // operands, columns on their way or in use
    static constexpr int K = 0, Q = K + 2 * K_BYTES, COLS = Q + STAGES * Q_BYTES;
    static constexpr int RED = COLS + CSTAGES * static_cast<int>(sizeof(Columns));   // f32 [2][KEYS]
    static constexpr int BAR = RED + 2 * KEYS * 4;
    enum { KFULL, KEMPTY, QFULL, QEMPTY = QFULL + STAGES, CFULL = QEMPTY + STAGES, CEMPTY = CFULL + CSTAGES,
           SFULL = CEMPTY + CSTAGES, SEMPTY = SFULL + 4, DRAIN = SEMPTY + 4, NBAR };
    static constexpr int TMEM_AT = BAR + NBAR * 8, BYTES = TMEM_AT + 16 + 1024;
    static_assert(BYTES <= 227 * 1024 && Q % 1024 == 0 && COLS % 16 == 0 && BAR % 8 == 0, "shared memory");
};
constexpr int MANY_THREADS = 768;   // products, row operands and two idle warps; widening; 4 x 4 of sums

__device__ __forceinline__ long long first_tile(const AttendArgs& g, int start, int b)
{
    return static_cast<long long>(start) * g.group / MOST_ROWS + b;
}

template <int D, typename T>
__global__ void __launch_bounds__(256) kv_weigh_rows_kernel(const WeighArgs w)
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
    const int pos = max(g.c.length[b], 0) - last + r;
    for (int h = threadIdx.x / 32; h < g.heads; h += 8) {
        const int row = (r - first) * g.group + h % g.group;
        uint8_t* record = w.operands +
                          (h / g.group * w.tiles + first_tile(g, first, b) + row / MOST_ROWS) * static_cast<long long>(C::RECORD);
        put_row<D, T>(g, static_cast<const T*>(g.q.data) + r * g.q.tok + h * g.q.head, g.stats[static_cast<size_t>(r) * g.heads + h],
                      pos, record, MOST_ROWS, row % MOST_ROWS, C::KB * MOST_ROWS, reinterpret_cast<Columns*>(record + C::Q_BYTES), lane);
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
    if (!unit_of(w, blockIdx.x % units, u))
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
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(C::SFULL + i), 1);
            mbar_init(bar(C::SEMPTY + i), 4);
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
                ok = warp_wait(w, bar(C::QFULL + stage), step / C::STAGES & 1);
                for (int k = 0; ok && k < 2; ++k) {
                    const int s = 2 * k + step % 2;
                    ok = warp_wait(w, bar(C::SEMPTY + s), (step / 2 & 1) ^ 1);
                    if (!ok)
                        break;
                    tc_fence_after();
                    product<D, C::PARTS>(lead, tmem + s * MOST_ROWS, sbase + C::K + k * C::K_BYTES,
                                         sbase + C::Q + stage * C::Q_BYTES, C::BLOCK, idesc);
                    umma_commit_by(lead, bar(C::SFULL + s));
                }
                if (ok)
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
        const uint8_t* records = w.operands + (static_cast<long long>(u.head) * w.tiles + first_tile(g, u.first, u.b)) * C::RECORD;
        for (int group = part; ok && group < groups; group += w.parts) {
            int lo, hi;
            range(group, lo, hi);
            for (int tile = lo; tile < hi; ++tile, ++step) {
                const int stage = step % C::STAGES, cstage = step % C::CSTAGES;
                ok = warp_wait(w, bar(C::QEMPTY + stage), (step / C::STAGES & 1) ^ 1) &&
                     warp_wait(w, bar(C::CEMPTY + cstage), (step / C::CSTAGES & 1) ^ 1);
                if (!ok)
                    break;
                if (lane == 0) {
                    const uint8_t* src = records + static_cast<long long>(tile) * C::RECORD;
                    fence_proxy_async_smem();   // the columns were read with ordinary loads
                    mbar_arrive_expect_tx(bar(C::QFULL + stage), C::Q_BYTES);
#pragma unroll
                    for (int i = 0; i < C::Q_BYTES; i += C::BLOCK)
                        bulk_g2s(sbase + C::Q + stage * C::Q_BYTES + i, src + i, C::BLOCK, bar(C::QFULL + stage));
                    mbar_arrive_expect_tx(bar(C::CFULL + cstage), sizeof(Columns));
                    bulk_g2s(sbase + C::COLS + cstage * sizeof(Columns), src + C::Q_BYTES, sizeof(Columns), bar(C::CFULL + cstage));
                }
            }
        }
        if (lane == 0) {   // the last fill of each stage lands before the CTA ends
            for (int i = max(0, step - C::STAGES); i < step; ++i)
                mbar_drain_wait(bar(C::QFULL + i % C::STAGES), i / C::STAGES & 1, WAIT_LIMIT_NS, g.wc.err);
            for (int i = max(0, step - C::CSTAGES); i < step; ++i)
                mbar_drain_wait(bar(C::CFULL + i % C::CSTAGES), i / C::CSTAGES & 1, WAIT_LIMIT_NS, g.wc.err);
        }
        __syncwarp();
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
        const int s = warp / 4 - 2, k = s / 2, odd = s % 2, t = threadIdx.x % KEYS;   // half of the keys, parity of the steps
        const uint32_t s_at = tmem + s * MOST_ROWS + (static_cast<uint32_t>(t & ~31) << 16);
        float* red = reinterpret_cast<float*>(smem + C::RED) + k * KEYS + t;
        for (int group = part; group < groups; group += w.parts) {
            int lo, hi;
            range(group, lo, hi);
            const int k0 = group * GROUP + k * KEYS, key = k0 + t;
            float2 sum = make_float2(0.0f, 0.0f);
            for (int tile = lo; ok && tile < hi; ++tile, ++step) {
                if (step % 2 != odd)
                    continue;
                const int cstage = step % C::CSTAGES;
                const Columns* cols = reinterpret_cast<const Columns*>(smem + C::COLS) + cstage;
                const int row0 = tile * MOST_ROWS, n = min(MOST_ROWS, u.rows - row0);
                ok = warp_wait(w, bar(C::CFULL + cstage), step / C::CSTAGES & 1) && warp_wait(w, bar(C::SFULL + s), step / 2 & 1);
                if (!ok)
                    break;
                tc_fence_after();
                const bool plain = n % 4 == 0 && all_seen(g, u.pos0 + row0 / g.group, u.pos0 + (row0 + n - 1) / g.group, k0, KEYS);
                for (int c = 0; c < n; c += 16) {
                    float x[16];
                    tmem_ld16_wait(s_at + c, x);
                    if (c + 16 >= n) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(bar(C::SEMPTY + s));
                    }
                    if (plain)
                        add_columns<false>(g, x, cols, c, n, key, sum);
                    else
                        add_columns<true>(g, x, cols, c, n, key, sum);
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(C::CEMPTY + cstage));
            }
            // the sums of odd steps to those of even ones
            if (odd)
                *red = sum.x + sum.y;
            ok = named_bar_and(2 + k, 256, ok);
            if (!ok)
                break;
            if (!odd && key < u.length) {
                const int page = u.table[key / KV_PAGE];
                if (page >= 0 && page < g.c.num_pages) {
                    const size_t at = (static_cast<size_t>(page) * g.c.kv_heads + u.head) * KV_PAGE + key % KV_PAGE;
                    w.out[at] = (key < u.pos0 ? w.decay * w.in[at] : 0.0f) + ((sum.x + sum.y) + *red);
                } else {
                    *g.c.bad = 1u;
                }
            }
            if (group + w.parts < groups)
                named_bar_sync(2 + k, 256);   // both have what they need of this group's
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        tmem_dealloc(tmem, 512);
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
    if (a.tiles == 0) {
        using C = Few<D, T>;
        static std::atomic<uint64_t> done{0};
        cudaError_t e = kv_allow_smem(kv_weigh_few_kernel<D, T>, C::bytes(MOST_ROWS) > 116 * 1024 ? C::bytes(MOST_ROWS) : 116 * 1024, &done);
        if (e != cudaSuccess)
            return e;
        // no more CTAs to an SM than its 512 columns of tensor memory are enough for
        const int resident = 512 / (2 * C::columns(a.cols));
        int bytes = C::bytes(a.cols);
        const int least = 227 * 1024 / (resident + 1);
        bytes = bytes > least ? bytes : least;
        const long long tiles = (keys + KEYS - 1) / KEYS, slots = 152ll * (227 * 1024 / (bytes + 1024));
        // the chip once over, or CTAs of 16 steps where lengths are uneven
        const long long even = slots / units, uneven = tiles / 16;
        a.parts = parts(tiles, even > uneven ? even : uneven);
        count_launch();
        return launch_dependent_smem(kv_weigh_few_kernel<D, T>, dim3(static_cast<unsigned int>(units * a.parts)),
                                     dim3(FEW_WARPS * 32), static_cast<size_t>(bytes), s, a);
    }
    using C = Many<D, T>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = kv_allow_smem(kv_weigh_many_kernel<D, T>, C::BYTES, &done);
    if (e != cudaSuccess)
        return e;
    count_launch();
    if ((e = launch_dependent(kv_weigh_rows_kernel<D, T>, dim3(static_cast<unsigned int>(a.a.ntok)), dim3(256), s, a)) != cudaSuccess)
        return e;
    const long long groups = (keys + 2 * KEYS - 1) / (2 * KEYS);
    a.parts = parts(groups, groups);
    count_launch();
    return launch_dependent_smem(kv_weigh_many_kernel<D, T>, dim3(static_cast<unsigned int>(units * a.parts)),
                                 dim3(MANY_THREADS), C::BYTES, s, a);
}

}  // namespace

size_t weigh_bytes(int dtype, int heads, int kv_heads, int dim, int batch, int ntok, int max_q, int* cols, long long* tiles)
{
    const long long group = heads / kv_heads, rows = (max_q < ntok ? max_q : ntok) * group;
    *cols = static_cast<int>(rows < 16 ? 16 : rows > MOST_ROWS ? MOST_ROWS : (rows + 15) / 16 * 16);
    *tiles = rows <= MOST_ROWS ? 0 : static_cast<long long>(ntok) * group / MOST_ROWS + batch + 1;
    const size_t record = static_cast<size_t>(dtype == KV_F32 ? 2 : 1) * MOST_ROWS * dim * 2 + sizeof(Columns);
    return static_cast<size_t>(*tiles) * kv_heads * record;
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

}  // namespace mmq
