// kv_prompt.cu -- attention over the 4-bit cache for many rows per sequence: prompts and
// their chunks, on the tensor cores.
//
//   S = Q K^T,  P = 2^(scale log2(e) S - ref),  O += P V,  o = O / sum P
//
// A CTA takes 256 rows (a row is a query token and one of the heads that share the kv
// head) as two tiles of 128 TMEM lanes, and walks the visible pages 128 keys at a time.
// The cached values are widened to f16, exactly, by one warpgroup for both tiles: K as
// [key][value] and V transposed as [value][key], the K-major operand tiles of the two
// products.  Q is scaled per row by a power of two (f16 rows are operands as they are) and
// split q = hi + lo in f16, P likewise: f32 rows use both parts (four products a tile,
// 22-bit operands), 16-bit rows are exact in hi (bf16 to 2^-24 of the row's largest) and
// round P to f16.
//
// TMEM: S of each tile in 128 columns, its P over the S that it came from (per 32 keys 16
// columns of hi and 16 of lo), O in D columns.  The tiles alternate on the tensor pipe, P V
// and the next Q K^T of one while the other's softmax runs: two threads a row read S, keep
// the row's reference and sums, and write P.  A row's O is rescaled only when its reference
// moves, which the lag of kv.cuh makes rare, by the softmax thread itself: its S arrived
// behind the last P V of the tile, so O is at rest.
//
// Where a CTA has 128 rows or fewer, both tiles hold them and take every other step, and
// their sums are joined at the end.
//
// 24 warps: warp 0 issues the MMAs, warp 1 copies the pages' bytes into a ring, warps 4-7
// widen, warps 8-15 and 16-23 are the softmax of tiles 0 and 1: two threads a row, one for
// each page of the step, which tell each other their largest x (with one thread a row the
// softmax took 2000 of a step's 3500 cycles, the products waiting for it).  Every wait is
// bounded; on expiry the roles leave their loops, copies and MMAs in flight are waited for,
// TMEM is freed and the CTA ends.
//
// What bounds it: a tile's chain of softmax, P V and Q K^T, which the other tile covers only
// in part; the tensor pipe is active in 60 % of the cycles (f32 rows: 52 %).  The f32 builds spill
// (0.6 % of the instructions executed), the others a word of 128-value heads at most.  On GB300:
// chunks of 2048 and 1944 bf16 tokens on 16384 and 13563, 32 heads of 128 on 8, 748 us, 1224
// TFLOP/s of the two products (a large library product reaches 1913); a prompt of 3314 f32
// tokens, 32 heads of 128, 161 us, 1.1 PFLOP/s of the four.
//
// Sums in TMEM are f32, but cut toward zero by every product: 16 a step for f32 rows, which
// cost values of one sign 1.4e-4 of the result after 20000 keys.  So f32 rows move O out
// every RUN steps and add it, rounded, to sums that lie in the rows of the result (or of
// their part), which belong to the CTA; L2 holds them.  What is left is the cut of RUN
// steps, below 1e-5 for such values (12 steps: 1.0e-5, 16: 1.3e-5) and up to 2e-5 where a first
// key outweighs the others, as each of its 160 products may cut 2^-23.  A step's weights are
// summed up over those steps too before they are added to the rest.  2048 tokens on 16384,
// 32 heads on 8, took 751 us for 648 without, and take 757 now.  What costs is the moves' bytes: moving every
// 8 steps took 770, without its loads and stores 666, and 818 when each CTA moved at steps
// of its own.  16-bit rows do without: their parts end before the cut passes their own
// rounding.
#include <type_traits>

#include "kv.cuh"

namespace mmq {
namespace {

constexpr int THREADS = 768;
constexpr int TILE = 128;                    // rows of a tile, keys of a step
constexpr int ROWS = KV_PROMPT_ROWS;
static_assert(ROWS == 2 * TILE, "two tiles");
constexpr int WIDEN_WARP = 4, SOFT_WARP = 8;
constexpr int SOFT_WARPS = 16;
// The launch's 80 registers a thread, shared out by warpgroup.
constexpr int LAUNCH_REGS = 80, CTRL_REGS = 24, WIDEN_REGS = 72, SOFT_REGS = 96;
static_assert(CTRL_REGS + WIDEN_REGS + 4 * SOFT_REGS == 6 * LAUNCH_REGS, "register split");
// .dec may only lower a warp's count and .inc only raise it (the other way is no instruction)
static_assert(CTRL_REGS < LAUNCH_REGS && WIDEN_REGS < LAUNCH_REGS && SOFT_REGS > LAUNCH_REGS, "register split");
constexpr int JOIN_BAR = 9;   // named barrier of all softmax warps (1-8: pairs)
constexpr int TILE_BAR = 10;  // of tile 1's
constexpr int RUN = 10;       // steps of a tile that O sums up before f32 rows move its sums out
constexpr int META = 8;   // steps whose page descriptions are kept: more than any role runs ahead

// HL: hi and lo parts of Q and P.
template <int D, bool HL>
struct Cfg {
    static constexpr int KB = D / 64;                            // 64-value blocks of a row
    static constexpr int PARTS = HL ? 2 : 1;
    static constexpr int BLOCK = TILE * 128;                     // 128 rows x 64 f16
    static constexpr int Q_BYTES = 2 * PARTS * KB * BLOCK;       // [tile][part][kb]
    static constexpr int K_BYTES = KB * BLOCK;                   // [kb][key]
    static constexpr int V_BYTES = 2 * D * 128;                  // [64 keys][value]
    static constexpr int BUFS = HL && D == 128 ? 1 : 2;          // buffers of each
    static constexpr int HALF = 36 * D;                          // bytes of a piece's K or V
    static constexpr int STAGE = 2 * HALF;                       // K or V of two pages
    static constexpr int STAGES = D == 128 ? 3 : 4;
    static constexpr int COLS = D == 64 && !HL ? 16 : 32;        // values of a row that a warp stages at a time
    static constexpr int STAGED = COLS * 4 + 16;                 // bytes of a staged row
    static_assert(16 * 32 * STAGED <= Q_BYTES + BUFS * K_BYTES, "staged rows of both tiles");
    static_assert(8 * 32 * STAGED + TILE * D * 4 <= Q_BYTES + BUFS * K_BYTES, "staged rows beside tile 1's sums");
    static constexpr int Q = 0;
    static constexpr int K = Q + Q_BYTES;
    static constexpr int V = K + BUFS * K_BYTES;
    static constexpr int RING = V + BUFS * V_BYTES;
    static constexpr int META_AT = RING + STAGES * STAGE;        // int2 [META]: tokens held of each page, -1 no page
    static constexpr int RED = META_AT + META * 8;               // f32 [2][page][row]: what a row's threads tell
    static constexpr int JOIN = RED + 2 * 2 * ROWS * 4;          // each other; float2 [row]: tile 1's {reference, sum}
    static constexpr int BAR = JOIN + TILE * 8;
    enum { QFULL, RFULL, REMPTY = RFULL + STAGES, KFULL = REMPTY + STAGES, KEMPTY = KFULL + BUFS,
           VFULL = KEMPTY + BUFS, VEMPTY = VFULL + BUFS, SFULL = VEMPTY + BUFS, PFULL = SFULL + 2,
           OFULL = PFULL + 2, DRAIN = OFULL + 2, NBAR };
    static constexpr int TMEM_AT = BAR + NBAR * 8;
    static constexpr int UNIT_AT = TMEM_AT + 4;                  // int: sequence, tile
    static constexpr int BYTES = UNIT_AT + 12 + 1024;            // and the alignment to 1024
    static_assert(BYTES <= 227 * 1024, "shared memory");
    static_assert(K % 1024 == 0 && V % 1024 == 0 && RING % 16 == 0 && META_AT % 8 == 0, "alignment");
};

constexpr uint32_t S_COL = 0, O_COL = 256;   // tile w: S at 128 w, O at 256 + D w

// 64 columns, both halves on their way at once: a load's latency, some 250 cycles beside the
// tensor cores' own traffic, is paid once.
__device__ __forceinline__ void tmem_load64(uint32_t taddr, uint32_t (&r)[2][32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0][0]), "=r"(r[0][1]), "=r"(r[0][2]), "=r"(r[0][3]), "=r"(r[0][4]), "=r"(r[0][5]), "=r"(r[0][6]), "=r"(r[0][7]), "=r"(r[0][8]), "=r"(r[0][9]), "=r"(r[0][10]), "=r"(r[0][11]), "=r"(r[0][12]), "=r"(r[0][13]), "=r"(r[0][14]), "=r"(r[0][15]), "=r"(r[0][16]), "=r"(r[0][17]), "=r"(r[0][18]), "=r"(r[0][19]), "=r"(r[0][20]), "=r"(r[0][21]), "=r"(r[0][22]), "=r"(r[0][23]), "=r"(r[0][24]), "=r"(r[0][25]), "=r"(r[0][26]), "=r"(r[0][27]), "=r"(r[0][28]), "=r"(r[0][29]), "=r"(r[0][30]), "=r"(r[0][31]), "=r"(r[1][0]), "=r"(r[1][1]), "=r"(r[1][2]), "=r"(r[1][3]), "=r"(r[1][4]), "=r"(r[1][5]), "=r"(r[1][6]), "=r"(r[1][7]), "=r"(r[1][8]), "=r"(r[1][9]), "=r"(r[1][10]), "=r"(r[1][11]), "=r"(r[1][12]), "=r"(r[1][13]), "=r"(r[1][14]), "=r"(r[1][15]), "=r"(r[1][16]), "=r"(r[1][17]), "=r"(r[1][18]), "=r"(r[1][19]), "=r"(r[1][20]), "=r"(r[1][21]), "=r"(r[1][22]), "=r"(r[1][23]), "=r"(r[1][24]), "=r"(r[1][25]), "=r"(r[1][26]), "=r"(r[1][27]), "=r"(r[1][28]), "=r"(r[1][29]), "=r"(r[1][30]), "=r"(r[1][31])
        : "r"(taddr), "r"(taddr + 32)
        : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&d);
}

// What a CTA works on; the same in every thread.
struct Unit {
    int b, head, split;
    int first, ntok, length;                 // the sequence's rows and tokens
    int row0, nrow;                          // rows row0 .. row0 + nrow - 1 of it
    int pos0;                                // position of the sequence's first new token
    int kend, nsink, page_lo, npage;         // keys [0, kend); pages 0 .. nsink - 1, page_lo ..
    int i0, steps;                           // first page of this split's and its 128-key steps
};
__device__ __forceinline__ int page_of(const Unit& u, int i) { return i < u.nsink ? i : u.page_lo + i - u.nsink; }

__device__ __forceinline__ bool wait(const AttendArgs& g, uint32_t bar, uint32_t parity)
{
    return mbar_wait_asleep(bar, parity, g.wc.limit_ns, g.wc.err);
}
__device__ __forceinline__ bool warp_wait(const AttendArgs& g, uint32_t bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, wait(g, bar, parity));
}

// For f32 rows a function of its own: inlined, more of the softmax was spilled (165 us for 161 on
// the prompt of 3314 tokens).
template <int D, typename T>
__device__ __noinline__ void clear_others_apart(const AttendArgs g)
{
    kv_clear_others<D, T>(g, 1ll << 60);
}

template <int D, typename T>
__global__ void __launch_bounds__(THREADS, 1) kv_prompt_kernel(const AttendArgs g)
{
    constexpr bool HL = sizeof(T) == 4;
    using C = Cfg<D, HL>;
    using P = Piece<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t sbase = raw + pad;
    // the shuffle tells the compiler that a warp's role is one for all its lanes
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    auto bar = [&](int i) -> uint32_t { return sbase + C::BAR + 8u * static_cast<uint32_t>(i); };

    grid_dep_wait();
    if (blockIdx.x == gridDim.x - 1) {
        if constexpr (HL)
            clear_others_apart<D, T>(g);
        else
            kv_clear_others<D, T>(g, 1ll << 60);   // the tiles take any number of new tokens
        return;
    }
    // ---------------------------------------------------------------- the unit
    // blocks run from the last row tile of the batch to the first (a sequence's later tiles
    // see more keys), all heads and splits of a tile together
    Unit u;
    int id = blockIdx.x;
    u.split = id % g.nsplit;
    id /= g.nsplit;
    u.head = id % g.c.kv_heads;
    id /= g.c.kv_heads;
    {
        // sequence b has ceil(rows / 256) tiles; the warp sums 32 sequences at a time
        const int want = g.row_tiles - 1 - id;
        int before = 0;
        u.first = u.ntok = u.length = 0;
        u.b = -1;
        u.row0 = 0;
        for (int b0 = 0; b0 < g.c.batch; b0 += 32) {
            int tiles = 0, s = 0, e = 0, len = 0;
            if (b0 + lane < g.c.batch) {
                s = g.c.start[b0 + lane];
                e = g.c.start[b0 + lane + 1];
                len = g.c.length[b0 + lane];
                if (s >= 0 && e > s && e <= g.ntok)
                    tiles = static_cast<int>((static_cast<long long>(e - s) * g.group + ROWS - 1) / ROWS);
            }
            int sum = tiles;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, d);
                sum += lane >= d ? v : 0;
            }
            const uint32_t here = __ballot_sync(0xffffffffu, want < before + sum);
            if (here) {
                const int l = __ffs(here) - 1;
                u.b = b0 + l;
                u.row0 = (want - before - __shfl_sync(0xffffffffu, sum - tiles, l)) * ROWS;
                u.first = __shfl_sync(0xffffffffu, s, l);
                u.ntok = __shfl_sync(0xffffffffu, e, l) - u.first;
                u.length = __shfl_sync(0xffffffffu, len, l);
                break;
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    if (u.b < 0)
        return;   // fewer tiles than the host's bound
    u.nrow = min(ROWS, u.ntok * g.group - u.row0);
    u.pos0 = max(u.length, 0) - u.ntok;
    {
        const int room = g.c.max_pages * KV_PAGE;
        const int plo = u.pos0 + u.row0 / g.group, phi = u.pos0 + (u.row0 + u.nrow - 1) / g.group;
        u.kend = min(max(phi + 1, 0), room);
        if (threadIdx.x == 0 && phi + 1 > room)
            *g.c.bad = 1u;
        const int klo = g.window > 0 ? min(max(plo - g.window + 1, 0), u.kend) : 0;
        u.page_lo = klo / KV_PAGE;
        u.nsink = min((min(g.sinks, u.kend) + KV_PAGE - 1) / KV_PAGE, u.page_lo);
        u.npage = u.nsink + (u.kend + KV_PAGE - 1) / KV_PAGE - u.page_lo;
        // a part is an even number of pages; the last takes what max_kv did not foresee
        const long long part0 = static_cast<long long>(u.split) * g.part_pages;
        u.i0 = static_cast<int>(min(part0, static_cast<long long>(u.npage)));
        u.steps = ((u.split == g.nsplit - 1 ? u.npage - u.i0 : min(g.part_pages, u.npage - u.i0)) + 1) / 2;
    }
    const bool two = u.nrow > TILE;        // else both tiles hold the same rows
    const int stride = two ? 1 : 2;        // and take every other step

    // ---------------------------------------------------------------- setup
    if (threadIdx.x == 0) {
        mbar_init(bar(C::QFULL), SOFT_WARPS);
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(bar(C::RFULL + i), 1);
            mbar_init(bar(C::REMPTY + i), 4);
        }
        for (int i = 0; i < C::BUFS; ++i) {
            mbar_init(bar(C::KFULL + i), 4);
            mbar_init(bar(C::KEMPTY + i), 1);
            mbar_init(bar(C::VFULL + i), 4);
            mbar_init(bar(C::VEMPTY + i), 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(bar(C::SFULL + w), 1);
            mbar_init(bar(C::PFULL + w), 8);
            mbar_init(bar(C::OFULL + w), 1);
        }
        mbar_init(bar(C::DRAIN), 1);
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(sbase + C::TMEM_AT, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<const uint32_t*>(smem + C::TMEM_AT);

    if (warp < WIDEN_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(CTRL_REGS));
        if (warp == 0) {
            // -------------------------------------------------------- MMA issue
            // the whole warp walks the loop, one lane's instructions take effect: descriptors
            // and addresses then stay in uniform registers
            const uint32_t lead = elect_one();
            constexpr uint32_t qk = idesc_f16_f32(TILE, TILE), pv = idesc_f16_f32(TILE, D);
            auto product_qk = [&](int w, int buf) {
#pragma unroll
                for (int part = C::PARTS - 1; part >= 0; --part)   // lo first: the sums are cut toward zero,
#pragma unroll                                                 // by less while they are small
                    for (int kb = 0; kb < C::KB; ++kb) {
                        const uint64_t a =
                            sdesc_k_sw128(sbase + C::Q + ((two || !HL ? w * C::PARTS : 0) + part) * C::KB * C::BLOCK + kb * C::BLOCK);
                        const uint64_t b = sdesc_k_sw128(sbase + C::K + buf * C::K_BYTES + kb * C::BLOCK);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f16_by(lead, tmem + S_COL + TILE * w, a + 2u * kk, b + 2u * kk, qk,
                                        (part < C::PARTS - 1 || kb || kk) ? 1u : 0u);
                    }
                umma_commit_by(lead, bar(C::SFULL + w));
            };
            auto product_pv = [&](int w, int buf, bool add) {
#pragma unroll
                for (int part = 0; part < C::PARTS; ++part)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {   // 32 keys
                        const uint64_t b = sdesc_k_sw128(sbase + C::V + buf * C::V_BYTES + c / 2 * D * 128);
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk)
                            umma_f16_ts_by(lead, tmem + O_COL + D * w,
                                           tmem + S_COL + TILE * w + 32 * c + 16 * part + 8 * kk,
                                           b + 4u * (c % 2) + 2u * kk, pv, (part | c | kk || add) ? 1u : 0u);
                    }
            };
            // a tile's steps are stride apart; K and V are free once the last tile that reads them has
            bool ok = u.steps == 0 || warp_wait(g, bar(C::QFULL), 0);
            auto ready_k = [&](int j) {
                ok = ok && warp_wait(g, bar(C::KFULL + j % C::BUFS), j / C::BUFS & 1);
                tc_fence_after();
            };
            for (int w = 0; w < 2; ++w) {
                const int j = two ? 0 : w;
                if (ok && j < u.steps) {
                    if (w == 0 || !two)
                        ready_k(j);
                    if (ok)
                        product_qk(w, j % C::BUFS);
                    if (w == 1 || !two)
                        umma_commit_by(lead, bar(C::KEMPTY + j % C::BUFS));
                }
            }
            for (int j = 0; ok && j < u.steps; ++j) {
                const int buf = j % C::BUFS, jn = j + stride, next = jn % C::BUFS;
                // with two buffers and both tiles at a step the next K is there before P is; else it
                // may be widened only after this step's products
                const bool early = C::BUFS == 2 && two;
                ok = warp_wait(g, bar(C::VFULL + buf), j / C::BUFS & 1);
                if (early && jn < u.steps)
                    ready_k(jn);
                for (int w = two ? 0 : j % 2; ok && w < (two ? 2 : j % 2 + 1); ++w) {
                    ok = warp_wait(g, bar(C::PFULL + w), j / stride & 1);
                    if (!ok)
                        break;
                    tc_fence_after();
                    product_pv(w, buf, HL ? j / stride % RUN != 0 : j >= stride);
                    if (w == 1 || !two)
                        umma_commit_by(lead, bar(C::VEMPTY + buf));
                    if (jn >= u.steps) {
                        umma_commit_by(lead, bar(C::OFULL + w));
                        continue;
                    }
                    if (!early && (w == 0 || !two))
                        ready_k(jn);
                    if (!ok)
                        break;
                    product_qk(w, next);
                    if (w == 1 || !two)
                        umma_commit_by(lead, bar(C::KEMPTY + next));
                }
            }
            umma_commit_by(lead, bar(C::DRAIN));   // nothing of this CTA's is left on the tensor pipe
            if (lead)
                mbar_drain_wait(bar(C::DRAIN), 0, WAIT_LIMIT_NS, g.wc.err);
        } else if (warp == 1) {
            // -------------------------------------------------------- page bytes: K, V of each step
            const int* table = g.c.table + static_cast<size_t>(u.b) * g.c.max_pages;
            int ids = -1, count = 0;
            // verification only: the fill of kv head 0's first rows that is left out (never armed,
            // never copied), so that the wait for it runs out
            const int skip = u.head == 0 && u.split == 0 && u.row0 == 0 ? g.wc.withhold_fill : -1;
            for (int j = 0; j < u.steps; ++j) {
                if (j % 16 == 0) {   // 32 page ids at a time, one per lane
                    const int i = u.i0 + 2 * j + lane;
                    ids = -1;
                    if (i < u.npage) {
                        ids = table[page_of(u, i)];
                        if (ids < 0 || ids >= g.c.num_pages) {
                            *g.c.bad = 1u;
                            ids = -1;
                        }
                    }
                }
                const int p0 = __shfl_sync(0xffffffffu, ids, j % 16 * 2);
                const int p1 = __shfl_sync(0xffffffffu, ids, j % 16 * 2 + 1);
                bool ok = true;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++count) {
                    const int stage = count % C::STAGES;
                    ok = warp_wait(g, bar(C::REMPTY + stage), (count / C::STAGES & 1) ^ 1);
                    if (!ok)
                        break;
                    if (lane == 0 && count != skip) {
                        int2* meta = reinterpret_cast<int2*>(smem + C::META_AT) + j % META;
                        if (kv == 0) {
                            const int i = u.i0 + 2 * j;
                            const int h0 = u.kend - page_of(u, i) * KV_PAGE, h1 = u.kend - page_of(u, i + 1) * KV_PAGE;
                            *meta = make_int2(p0 < 0 ? -1 : min(h0, KV_PAGE), p1 < 0 ? -1 : min(h1, KV_PAGE));
                        }
                        fence_proxy_async_smem();   // the stage was read with ordinary loads
                        mbar_arrive_expect_tx(bar(C::RFULL + stage), ((p0 >= 0) + (p1 >= 0)) * C::HALF);
                        const uint32_t dst = sbase + C::RING + stage * C::STAGE;
                        const size_t piece = static_cast<size_t>(g.c.kv_heads) * P::BYTES;
                        const uint8_t* src = g.c.pages + static_cast<size_t>(u.head) * P::BYTES + kv * C::HALF;
                        if (p0 >= 0)
                            bulk_g2s(dst, src + p0 * piece, C::HALF, bar(C::RFULL + stage));
                        if (p1 >= 0)
                            bulk_g2s(dst + C::HALF, src + p1 * piece, C::HALF, bar(C::RFULL + stage));
                    }
                }
                if (!ok)
                    break;
            }
            if (lane == 0)   // the last fill of each stage lands before the CTA ends
                for (int i = max(0, count - C::STAGES); i < count; ++i)
                    if (i != skip)
                        mbar_drain_wait(bar(C::RFULL + i % C::STAGES), i / C::STAGES & 1, WAIT_LIMIT_NS, g.wc.err);
        }
        __syncwarp();
    } else if (warp < SOFT_WARP) {
        // ------------------------------------------------------------ widening
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(WIDEN_REGS));
        const int t = threadIdx.x - WIDEN_WARP * 32;
        int count = 0;
        bool ok = true;
        for (int j = 0; ok && j < u.steps; ++j) {
            const int buf = j % C::BUFS;
            const uint32_t empty = (j / C::BUFS & 1) ^ 1;
            {   // K: a thread per key
                const int stage = count % C::STAGES;
                ok = warp_wait(g, bar(C::RFULL + stage), count / C::STAGES & 1) &&
                     warp_wait(g, bar(C::KEMPTY + buf), empty);
                if (!ok)
                    break;
                const int2 held = reinterpret_cast<const int2*>(smem + C::META_AT)[j % META];
                const bool there = (t < KV_PAGE ? held.x : held.y) >= 0;
                const uint8_t* src = smem + C::RING + stage * C::STAGE + t / KV_PAGE * C::HALF;
                uint8_t* dst = smem + C::K + buf * C::K_BYTES + t * 128;
#pragma unroll
                for (int gr = 0; gr < P::NG; ++gr) {
                    const uint4 v = *reinterpret_cast<const uint4*>(src + P::k_chunk(t % KV_PAGE, gr));
                    // a page that is not there gives zeros: any code times the scale 0
                    const uint16_t sc = *reinterpret_cast<const uint16_t*>(src + P::k_scale(t % KV_PAGE, gr));
                    const __half2 s = __half2half2(__ushort_as_half(there ? sc : 0));
                    const __half2 sb = kv_addend(s);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 o = make_uint4(kv_h2u(kv_widen<0>(w[i], s, sb)), kv_h2u(kv_widen<1>(w[i], s, sb)),
                                             kv_h2u(kv_widen<2>(w[i], s, sb)), kv_h2u(kv_widen<3>(w[i], s, sb)));
                        *reinterpret_cast<uint4*>(dst + gr / 2 * C::BLOCK + ((gr % 2 * 4 + i) ^ (t & 7)) * 16) = o;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(C::KFULL + buf));
                    mbar_arrive(bar(C::REMPTY + stage));
                }
                ++count;
            }
            {   // V: a thread per 8 keys (chunk c of a page's row) and 16 values
                const int stage = count % C::STAGES;
                ok = warp_wait(g, bar(C::RFULL + stage), count / C::STAGES & 1) &&
                     warp_wait(g, bar(C::VEMPTY + buf), empty);
                if (!ok)
                    break;
                const int2 meta = reinterpret_cast<const int2*>(smem + C::META_AT)[j % META];
                for (int item = t; item < 2 * 8 * (D / 16); item += 128) {
                    const int c = item % 8, a = item / 8 % (D / 16), h = item / 8 / (D / 16);
                    const int held = h ? meta.y : meta.x;
                    const uint8_t* src = smem + C::RING + stage * C::STAGE + h * C::HALF - P::V_CODES;
                    uint32_t w[4][4];
                    __half2 s[4], sb[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int pair = 4 * c + k;
                        const uint4 v = *reinterpret_cast<const uint4*>(src + P::v_chunk(pair, a));
                        w[k][0] = v.x, w[k][1] = v.y, w[k][2] = v.z, w[k][3] = v.w;
                        // slots without a token hold anything, and 0 times no number is none
                        uint32_t sc = *reinterpret_cast<const uint32_t*>(src + P::v_scale(pair, a / 2));
                        sc = 2 * pair + 1 < held ? sc : 2 * pair < held ? sc & 0xffffu : 0u;
                        s[k] = kv_u2h(sc);
                        sb[k] = kv_addend(s[k]);
                    }
                    uint8_t* dst = smem + C::V + buf * C::V_BYTES + h * D * 128 + 16 * a * 128;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        auto put = [&](int n, uint4 o) {
                            *reinterpret_cast<uint4*>(dst + (4 * i + n) * 128 + ((c ^ (4 * i + n) & 7) << 4)) = o;
                        };
                        put(0, make_uint4(kv_h2u(kv_widen<0>(w[0][i], s[0], sb[0])), kv_h2u(kv_widen<0>(w[1][i], s[1], sb[1])),
                                          kv_h2u(kv_widen<0>(w[2][i], s[2], sb[2])), kv_h2u(kv_widen<0>(w[3][i], s[3], sb[3]))));
                        put(1, make_uint4(kv_h2u(kv_widen<1>(w[0][i], s[0], sb[0])), kv_h2u(kv_widen<1>(w[1][i], s[1], sb[1])),
                                          kv_h2u(kv_widen<1>(w[2][i], s[2], sb[2])), kv_h2u(kv_widen<1>(w[3][i], s[3], sb[3]))));
                        put(2, make_uint4(kv_h2u(kv_widen<2>(w[0][i], s[0], sb[0])), kv_h2u(kv_widen<2>(w[1][i], s[1], sb[1])),
                                          kv_h2u(kv_widen<2>(w[2][i], s[2], sb[2])), kv_h2u(kv_widen<2>(w[3][i], s[3], sb[3]))));
                        put(3, make_uint4(kv_h2u(kv_widen<3>(w[0][i], s[0], sb[0])), kv_h2u(kv_widen<3>(w[1][i], s[1], sb[1])),
                                          kv_h2u(kv_widen<3>(w[2][i], s[2], sb[2])), kv_h2u(kv_widen<3>(w[3][i], s[3], sb[3]))));
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(C::VFULL + buf));
                    mbar_arrive(bar(C::REMPTY + stage));
                }
                ++count;
            }
        }
    } else {
        // ------------------------------------------------------------ softmax: two threads a row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(SOFT_REGS));
        const int w = (warp - SOFT_WARP) / 8, h = (warp - SOFT_WARP) / 4 % 2;   // tile, page of a step
        const int l = warp % 4 * 32 + lane;                                      // TMEM lane
        const int pair = 1 + 4 * w + warp % 4;   // named barrier of the two warps that share 32 rows
        float* red = reinterpret_cast<float*>(smem + C::RED) + TILE * w + l;     // [2][page]: ROWS apart
        const int tile0 = two ? TILE * w : 0;    // the tile's first row
        const bool mine = tile0 + l < u.nrow;
        const int row = u.row0 + min(tile0 + l, u.nrow - 1);
        const long long token = u.first + row / g.group;
        const int head = u.head * g.group + row % g.group;
        const long long q_at = token * g.q.tok + head * g.q.head;
        float coef = 1.0f;
        if (u.steps > 0) {
            // 2^-e q into the operand tiles, e the exponent of the row's largest magnitude.  The
            // warp loads 16 of its 32 rows, eight lanes a row (lanes past the last row load that
            // one again: their rows go nowhere)
            constexpr int LOADS = D / 32;                              // of four values a lane, four rows at once
            constexpr int BATCH = sizeof(T) == 4 && D == 128 ? 2 : 4;  // 32 registers of loads on their way
            const int sub = lane / 8, c = lane % 8 * 4;
            uint8_t* dst = smem + C::Q + w * C::PARTS * C::KB * C::BLOCK;
#pragma unroll 1
            for (int i0 = 16 * h; i0 < 16 * h + 16; i0 += 4 * BATCH) {
                Raw4<T> x[BATCH][LOADS];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const T* q = static_cast<const T*>(g.q.data) + __shfl_sync(0xffffffffu, q_at, i0 + 4 * k + sub) + c;
#pragma unroll
                    for (int i = 0; i < LOADS; ++i)
                        x[k][i].load(q + 32 * i, g.wide);
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int r32 = warp % 4 * 32 + i0 + 4 * k + sub;
                    int e = 0;
                    float f = 1.0f;
                    if constexpr (!std::is_same<T, __half>::value) {   // f16 is an operand as it is
                        float a = 0.0f;
#pragma unroll
                        for (int i = 0; i < LOADS; ++i) {
                            const float4 v = x[k][i].get();
                            a = fmaxf(a, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
                        }
#pragma unroll
                        for (int s = 1; s < 8; s <<= 1)
                            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, s));
                        e = kv_exponent(a);
                        f = kv_pow2(-e);
                    }
#pragma unroll
                    for (int i = 0; i < LOADS; ++i) {
                        const int d = 32 * i + c;
                        uint8_t* at = dst + d / 64 * C::BLOCK + r32 * 128 + ((d / 8 % 8 ^ (r32 & 7)) << 4) + d % 8 * 2;
                        if constexpr (std::is_same<T, __half>::value) {
                            *reinterpret_cast<uint2*>(at) = *reinterpret_cast<const uint2*>(x[k][i].e);
                        } else {
                            const float4 v = x[k][i].get();
                            uint2 hi, lo;
                            kv_split2(v.x * f, v.y * f, hi.x, lo.x);
                            kv_split2(v.z * f, v.w * f, hi.y, lo.y);
                            *reinterpret_cast<uint2*>(at) = hi;
                            if (HL)
                                *reinterpret_cast<uint2*>(at + C::KB * C::BLOCK) = lo;
                        }
                    }
                    if (c == 0)
                        red[r32 - l] = fminf(fmaxf(g.scale_log2 * kv_pow2(e), 1e-38f), 1e38f);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(C::QFULL));
        }
        named_bar_sync(pair, 64);
        if (u.steps > 0)
            coef = red[0];
        named_bar_sync(pair, 64);   // both have read theirs

        const uint32_t lanes = static_cast<uint32_t>(l & ~31) << 16;
        const uint32_t s_at = tmem + lanes + S_COL + TILE * w + 64 * h;
        const uint32_t o_at = tmem + lanes + O_COL + D * w + D / 2 * h;   // each thread has half of the row's O
        const int pos = mine ? u.pos0 + row / g.group : -1;
        // positions of the tile's rows, for steps that no mask touches
        const int plo = u.pos0 + (u.row0 + tile0) / g.group;
        const int phi = u.pos0 + (u.row0 + min(u.nrow, tile0 + TILE) - 1) / g.group;
        float ref = -INFINITY, sum = 0.0f;
        [[maybe_unused]] float moved_sum = 0.0f;   // f32 rows: of the steps whose O was moved out
        bool ok = true;
        int k = 0;   // steps of this tile so far

        // of the row's sums among the parts'; of its result
        auto part_row = [&] { return static_cast<long long>(u.split) * g.ntok * g.heads + token * g.heads + head; };
        auto result = [&] { return g.nsplit > 1 ? part_row() * D : token * g.out.tok + head * g.out.head; };
        // Sums moved out lie where the result will: in the warp's rows, its half of their values,
        // but four values of one lane after four of the next, so that a warp moves whole lines.
        // Tile 1, when it has tile 0's rows, keeps them in place of its own Q.
        constexpr int FOURS = D / 8;   // of four values a thread has
        float moved = 1.0f;            // what the moved sums' reference has come to since
        [[maybe_unused]] const bool inside = !two && w == 1;
        [[maybe_unused]] float4* const slots = reinterpret_cast<float4*>(smem + C::Q + C::Q_BYTES / 2) + h * TILE + l;
        [[maybe_unused]] const int valid = min(max(u.nrow - tile0 - (l & ~31), 0), 32);   // the warp's rows
        [[maybe_unused]] const bool wide = g.nsplit > 1 || g.wide;
        [[maybe_unused]] auto moved_to = [&](long long out_at, int i) {
            const int at = i * valid + lane;
            float* rows = g.nsplit > 1 ? g.part : static_cast<float*>(g.out.data);
            return rows + __shfl_sync(0xffffffffu, out_at, at / FOURS & 31) + D / 2 * h + at % FOURS * 4;
        };
        [[maybe_unused]] auto moved_load = [&](float4 (&x)[FOURS]) {
            const long long out_at = result();
#pragma unroll
            for (int i = 0; i < FOURS; ++i) {
                x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (inside) {
                    x[i] = slots[i * 2 * TILE];
                } else {
                    const float* p = moved_to(out_at, i);
                    if (lane < valid) {
                        Raw4<float> v;
                        v.load(p, wide);
                        x[i] = v.get();
                    }
                }
            }
        };
        // O added to the moved sums x
        [[maybe_unused]] auto move_out = [&](const float4 (&x)[FOURS]) {
            const long long out_at = result();
#pragma unroll
            for (int d = 0; d < D / 2; d += 16) {
                float o[16];
                tmem_ld16_wait(o_at + d, o);
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                    const int i = (d + c) / 4;
                    const float4 v = make_float4(fmaf(x[i].x, moved, o[c]), fmaf(x[i].y, moved, o[c + 1]),
                                                 fmaf(x[i].z, moved, o[c + 2]), fmaf(x[i].w, moved, o[c + 3]));
                    if (inside) {
                        slots[i * 2 * TILE] = v;
                    } else {
                        float* p = moved_to(out_at, i);
                        if (lane < valid)
                            store4(p, v, wide);
                    }
                }
            }
            moved_sum = fmaf(moved_sum, moved, sum);
            sum = 0.0f;
            moved = 1.0f;
        };
        // the moved sums x added to O
        [[maybe_unused]] auto move_in = [&](const float4 (&x)[FOURS]) {
#pragma unroll
            for (int d = 0; d < D / 2; d += 16) {
                float o[16];
                uint32_t v[16];
                tmem_ld16_wait(o_at + d, o);
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                    const float4 y = x[(d + c) / 4];
                    v[c] = __float_as_uint(fmaf(y.x, moved, o[c]));
                    v[c + 1] = __float_as_uint(fmaf(y.y, moved, o[c + 1]));
                    v[c + 2] = __float_as_uint(fmaf(y.z, moved, o[c + 2]));
                    v[c + 3] = __float_as_uint(fmaf(y.w, moved, o[c + 3]));
                }
                tmem_store16(o_at + d, v);
            }
            tmem_wait_st();
        };
        {
            for (int j = two ? 0 : w; j < u.steps; j += stride, ++k) {
                if (HL && k > 0 && k % RUN == 0) {
                    float4 x[FOURS] = {};
                    if (k > RUN)
                        moved_load(x);   // on its way while S is waited for
                    ok = warp_wait(g, bar(C::SFULL + w), k & 1);
                    tc_fence_after();
                    move_out(x);
                } else {
                    ok = warp_wait(g, bar(C::SFULL + w), k & 1);
                    tc_fence_after();
                }
                const int2 held = reinterpret_cast<const int2*>(smem + C::META_AT)[j % META];
                const int kbase = page_of(u, u.i0 + 2 * j + h) * KV_PAGE;
                const bool there = (h ? held.y : held.x) >= 0;
                const bool plain = there && kbase + KV_PAGE - 1 <= plo &&
                                   (g.window == 0 || kbase > phi - g.window || kbase + KV_PAGE <= g.sinks);

                // false: one of the two warps has given up
                auto softmax = [&](auto with_mask) {
                    uint32_t x[2][32];
                    tmem_load64(s_at, x);
                    if constexpr (decltype(with_mask)::value) {
                        const uint64_t seen = there ? kv_seen_bits(pos, kbase, g.window, g.sinks) : 0;
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            x[i / 32][i % 32] = seen >> i & 1u ? x[i / 32][i % 32] : 0xff800000u;   // -inf
                    }
                    float tops[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tops[c] = __uint_as_float(x[c / 2][c % 2 * 16]);
#pragma unroll
                        for (int i = 0; i < 16; i += 2)
                            tops[c] = fmaxf(tops[c], fmaxf(__uint_as_float(x[c / 2][c % 2 * 16 + i]),
                                                           __uint_as_float(x[c / 2][c % 2 * 16 + i + 1])));
                    }
                    float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    red[(2 * (k & 1) + h) * ROWS] = top;
                    if (!named_bar_and(pair, 64, ok))
                        return false;
                    top = fmaxf(top, red[(2 * (k & 1) + 1 - h) * ROWS]) * coef;
                    const bool raise = top > ref + KV_REF_LIMIT;   // also the first visible key
                    if (__any_sync(0xffffffffu, raise)) {
                        const float next = raise ? top - kv_ref_below<T>() : ref;
                        const float f = raise ? kv_ex2(ref - next) : 1.0f;
                        ref = next;
                        sum *= f;
                        moved *= f;
                        if (HL ? k % RUN != 0 : k > 0) {
#pragma unroll 1
                            for (int d = 0; d < D / 2; d += 16) {
                                float o[16];
                                uint32_t v[16];
                                tmem_ld16_wait(o_at + d, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    v[i] = __float_as_uint(o[i] * f);
                                tmem_store16(o_at + d, v);
                            }
                        }
                    }
                    const float base = ref == -INFINITY ? 0.0f : ref;
                    float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 e = ffma2(make_float2(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])),
                                             make_float2(coef, coef), make_float2(-base, -base));
                            e = make_float2(kv_ex2(e.x), kv_ex2(e.y));
                            part[i % 2] = fadd2(part[i % 2], e);
                            if (HL)
                                kv_split2(e.x, e.y, hi[i], lo[i]);
                            else
                                hi[i] = kv_h2u(__floats2half2_rn(e.x, e.y));
                        }
                        // P's keys go over columns of S that this thread has read
                        tmem_store16(s_at + 32 * c, hi);
                        if (HL)
                            tmem_store16(s_at + 32 * c + 16, lo);
                    }
                    sum += (part[0].x + part[0].y) + (part[1].x + part[1].y);
                    return true;
                };
                // two builds, so that steps without a mask carry no selects for it
                ok = plain ? softmax(std::false_type{}) : softmax(std::true_type{});
                if (!ok)
                    break;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(C::PFULL + w));
            }
            if (ok && k > 0) {
                if (HL && k > RUN) {
                    float4 x[FOURS];
                    moved_load(x);
                    warp_wait(g, bar(C::OFULL + w), 0);
                    tc_fence_after();
                    move_in(x);
                } else {
                    warp_wait(g, bar(C::OFULL + w), 0);
                    tc_fence_after();
                }
            }
        }
        if (HL)
            sum = fmaf(moved_sum, moved, sum);
        red[2 * ROWS * (k & 1) + h * ROWS] = sum;
        named_bar_sync(pair, 64);
        sum += red[2 * ROWS * (k & 1) + (1 - h) * ROWS];

        // with the same rows in both tiles, tile 0 takes over what tile 1 has: O by way of the shared
        // memory of Q and K, which no product reads any more
        float4* joined = reinterpret_cast<float4*>(smem + C::Q + 8 * 32 * C::STAGED) + h * TILE + l;   // [value / 4][page][row]
        float f_own = 1.0f, f_other = 0.0f;
        if (!two && u.steps > 1) {
            float2* other = reinterpret_cast<float2*>(smem + C::JOIN) + l;
            if (w == 1) {
                if (HL && u.steps > 2 * RUN)   // what was moved lies there too: every thread has its own back
                    named_bar_sync(TILE_BAR, SOFT_WARPS * 16);
#pragma unroll 1
                for (int d = 0; d < D / 2; d += 16) {
                    float o[16];
                    tmem_ld16_wait(o_at + d, o);
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        joined[(d + i) / 4 * 2 * TILE] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
                if (h == 0)
                    *other = make_float2(ref, sum);
            }
            named_bar_sync(JOIN_BAR, SOFT_WARPS * 32);
            const float2 v = *other;
            const float top = fmaxf(ref, v.x);
            f_own = ref == -INFINITY ? 0.0f : kv_ex2(ref - top);
            f_other = v.x == -INFINITY ? 0.0f : kv_ex2(v.x - top);
            sum = f_own * sum + f_other * v.y;
            ref = top;
        }
        if (w == 0 || two) {
            // half of a row's share of the result, by way of shared memory (the tile's Q is done
            // with): the warp writes four rows' 32 values at a time, whole lines for the strided 16
            // bytes a thread that its own row would take
            const float inv = g.nsplit > 1 ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
            const long long out_at = result();
            if (g.nsplit > 1 && mine && h == 0)
                g.part_ml[part_row()] = make_float2(ref, sum);
            constexpr int COLS = C::COLS, ROW = C::STAGED, LPR = COLS / 4;
            uint8_t* stage = smem + C::Q + (warp - SOFT_WARP) * 32 * ROW;
            const int sub = lane / LPR, c = lane % LPR * 4;
            long long to[LPR];   // of the rows whose values c .. c + 3 this lane writes
            uint32_t there = 0;
#pragma unroll
            for (int i = 0; i < LPR; ++i) {
                const int src = 32 / LPR * i + sub;
                to[i] = __shfl_sync(0xffffffffu, out_at, src) + c + D / 2 * h;
                there |= (__shfl_sync(0xffffffffu, mine, src) ? 1u : 0u) << i;
            }
#pragma unroll
            for (int d = 0; d < D / 2; d += COLS) {
                float o[COLS];
                if (u.steps > 0) {
#pragma unroll
                    for (int i = 0; i < COLS; i += 16)
                        tmem_ld16_wait(o_at + d + i, *reinterpret_cast<float(*)[16]>(o + i));
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < COLS; i += 4) {
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (u.steps > 0) {
                        v = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        if (!two && u.steps > 1) {
                            const float4 y = joined[(d + i) / 4 * 2 * TILE];
                            v = make_float4(f_own * v.x + f_other * y.x, f_own * v.y + f_other * y.y,
                                            f_own * v.z + f_other * y.z, f_own * v.w + f_other * y.w);
                        }
                        v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                    }
                    *reinterpret_cast<float4*>(stage + lane * ROW + i * 4) = v;
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < LPR; ++i) {
                    const float4 v = *reinterpret_cast<const float4*>(stage + (32 / LPR * i + sub) * ROW + c * 4);
                    if (there >> i & 1u) {
                        if (g.nsplit > 1)
                            *reinterpret_cast<float4*>(g.part + to[i] + d) = v;
                        else
                            store4(static_cast<T*>(g.out.data) + to[i] + d, v, g.wide);
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        tmem_dealloc(tmem, 512);
}

template <int D, typename T>
cudaError_t launch_prompt(const AttendArgs& a, cudaStream_t s)
{
    using C = Cfg<D, sizeof(T) == 4>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = kv_allow_smem(kv_prompt_kernel<D, T>, C::BYTES, &done);
    if (e != cudaSuccess)
        return e;
    // the register split draws on what the launch reserves: with fewer the softmax would
    // wait for registers that never come
    static std::atomic<int> regs{0};
    if (regs.load() == 0) {
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, kv_prompt_kernel<D, T>)) != cudaSuccess)
            return e;
        regs.store(fa.numRegs);
    }
    if (regs.load() != LAUNCH_REGS)
        return cudaErrorInvalidConfiguration;
    const unsigned int grid =
        static_cast<unsigned int>(static_cast<long long>(a.nsplit) * a.c.kv_heads * a.row_tiles + 1);
    count_launch();
    return launch_dependent_smem(kv_prompt_kernel<D, T>, dim3(grid), dim3(THREADS), C::BYTES, s, a);
}

}  // namespace

cudaError_t launch_kv_prompt(const AttendArgs& a, int dim, int dtype, cudaStream_t s)
{
    if (dim == 128)
        return dtype == KV_F32   ? launch_prompt<128, float>(a, s)
               : dtype == KV_F16 ? launch_prompt<128, __half>(a, s)
                                 : launch_prompt<128, __nv_bfloat16>(a, s);
    return dtype == KV_F32   ? launch_prompt<64, float>(a, s)
           : dtype == KV_F16 ? launch_prompt<64, __half>(a, s)
                             : launch_prompt<64, __nv_bfloat16>(a, s);
}

}  // namespace mmq
