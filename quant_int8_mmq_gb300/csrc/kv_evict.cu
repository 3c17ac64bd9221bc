// kv_evict.cu -- fewer tokens in the 4-bit cache: which stay, and their way to other pages.
//
// Of a sequence of n > keep tokens stay, per kv head, the first ones, the last ones, and of
// the rest the m with the largest weights (ties: the lower position).  The m-th largest weight
// T is found by a radix search: weights as unsigned numbers of the same order, four
// histograms of 8 bits of those that agree with T in the bits known so far.  A token
// then stays if its weight is above T, or equal and among the first of those that equal it, and
// its new place is the number of tokens before it that stay.
//
// kv_choose_kernel: a CTA, or a cluster of them for few long sequences, per (sequence, kv
// head), its weights in shared memory.  Bound by the latency of its rounds: loads through the page table,
// four times histogram, merge and search, then places; 131071 tokens of 8 kv heads in 23 us, 4
// sequences of up to 1280 in 8.  (With warp matches instead of shared-memory atomics 99 us for 37 with
// the move; all counts of a cluster's bins read by one thread each 48, a load from another CTA being
// 1000 cycles.)
//
// kv_move_kernel: a CTA gathers the 64 tokens of a new page and kv head, codes and scales, 16 bytes a
// thread; nothing is decoded, the two tokens that share a word of value codes are put together from the
// halves of theirs.  Bound by its gathers: three dependent loads (old place, page id, codes), of which two
// are on their way while the page before is moved; and words of values are two tokens', so that one that
// stays without its neighbour has twice its bytes read.  So as many warps as an SM has room for, at 32
// registers (at 57, half of them, 147 us for 125).  64 sequences of up to 8192 tokens to 4096, 8 heads of 128:
// 122 us for both kernels, 0.70 of a plain copy's rate on the bytes that stay.
#include <type_traits>

#include "kv.cuh"

namespace mmq {
namespace {

constexpr int BINS = 256, ROUNDS = 4;

// Unsigned numbers in the order of f32 ones; -0 as 0, no number below all others.
__device__ __forceinline__ uint32_t order_of(float w)
{
    const uint32_t u = __float_as_uint(w + 0.0f);
    return w != w ? 0u : u >> 31 ? ~u : u | 0x80000000u;
}

template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 3) kv_choose_kernel(const EvictArgs g)
{
    constexpr int CHOOSE = WARPS * 32;
    static_assert(WARPS >= KV_MAX_CLUSTER, "a warp fetches a CTA's bins");
    extern __shared__ __align__(16) uint32_t keys[];   // [g.held] of this CTA's tokens
    __shared__ __align__(16) uint32_t hist[ROUNDS][BINS];
    __shared__ uint2 counts[WARPS];             // tokens above T, and equal to it
    __shared__ uint2 mine;                             // of the CTA
    __shared__ __align__(16) uint32_t all[KV_MAX_CLUSTER][BINS];
    __shared__ uint2 found[ROUNDS];                    // bin, tokens above it
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    grid_dep_wait();
    grid_dep_launch();
    const int unit = blockIdx.x / g.cluster, rank = blockIdx.x % g.cluster;
    const int b = unit / g.c.kv_heads, head = unit % g.c.kv_heads;
    const int room = g.c.max_pages * KV_PAGE;
    const int n = min(max(g.c.length[b], 0), room);
    if (threadIdx.x == 0 && n != g.c.length[b])
        *g.c.bad = 1u;
    int* kept = g.kept + (static_cast<size_t>(b) * g.c.kv_heads + head) * g.keep;
    const int stay = min(n, g.keep);
    for (int i = stay + rank * CHOOSE + static_cast<int>(threadIdx.x); i < g.keep; i += g.cluster * CHOOSE)
        kept[i] = -1;
    if (n <= g.keep) {
        for (int i = rank * CHOOSE + threadIdx.x; i < n; i += g.cluster * CHOOSE)
            kept[i] = i;
        return;
    }

    // this CTA's tokens: whole pages, those past what it holds are read again each time
    const int pages = (n + KV_PAGE - 1) / KV_PAGE, share = (pages + g.cluster - 1) / g.cluster;
    const int lo = min(rank * share * KV_PAGE, n), hi = min(lo + share * KV_PAGE, n), size = hi - lo;
    const int* table = g.c.table + static_cast<size_t>(b) * g.c.max_pages;
    auto read = [&](int j) {   // the order of token lo + j
        const int page = table[(lo + j) / KV_PAGE];
        if (page < 0 || page >= g.c.num_pages) {
            *g.c.bad = 1u;
            return 0u;
        }
        return order_of(g.weights[(static_cast<size_t>(page) * g.c.kv_heads + head) * KV_PAGE + (lo + j) % KV_PAGE]);
    };
    const int inside = min(size, g.held), quads = (inside + 3) / 4;
    constexpr int BATCH = 4;
    for (int q0 = threadIdx.x; q0 < quads; q0 += BATCH * CHOOSE) {   // four weights a thread and load
        int page[BATCH];
        float4 v[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int q = q0 + i * CHOOSE;
            page[i] = q < quads ? table[lo / KV_PAGE + q / 16] : -1;
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int q = q0 + i * CHOOSE;
            v[i] = make_float4(NAN, NAN, NAN, NAN);
            if (page[i] >= 0 && page[i] < g.c.num_pages)
                v[i] = *reinterpret_cast<const float4*>(
                    g.weights + (static_cast<size_t>(page[i]) * g.c.kv_heads + head) * KV_PAGE + q % 16 * 4);
            else if (q < quads)
                *g.c.bad = 1u;
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int q = q0 + i * CHOOSE;
            if (q < quads)
                *reinterpret_cast<uint4*>(keys + 4 * q) =
                    make_uint4(order_of(v[i].x), order_of(v[i].y), order_of(v[i].z), order_of(v[i].w));
        }
    }
    for (int i = threadIdx.x; i < ROUNDS * BINS; i += CHOOSE)
        hist[i / BINS][i % BINS] = 0;
    __syncthreads();
    auto key = [&](int j) { return j < g.held ? keys[j] : read(j); };
    // tokens [from, to) compete for `need` places
    const int from = g.first, to = n - g.last;
    uint32_t need = static_cast<uint32_t>(g.keep - g.first - g.last);
    uint32_t prefix = 0, known = 0;
    for (int round = 0; need > 0 && round < ROUNDS; ++round) {
        const int shift = 24 - 8 * round;
        auto count = [&](uint32_t k, int j) {
            if (j < size && lo + j >= from && lo + j < to && (k & known) == prefix)
                atomicAdd(&hist[round][k >> shift & (BINS - 1)], 1u);
        };
        for (int q0 = 0; q0 < quads; q0 += CHOOSE) {
            const int q = q0 + threadIdx.x;
            const uint4 k = q < quads ? *reinterpret_cast<const uint4*>(keys + 4 * q) : make_uint4(0, 0, 0, 0);
            const int j = q < quads ? 4 * q : size;
            if (j + 3 < size && lo + j >= from && lo + j + 3 < to) {
                const uint32_t e[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if ((e[i] & known) == prefix)
                        atomicAdd(&hist[round][e[i] >> shift & (BINS - 1)], 1u);
            } else {
                count(k.x, j);
                count(k.y, j + 1);
                count(k.z, j + 2);
                count(k.w, j + 3);
            }
        }
        for (int j0 = g.held; j0 < size; j0 += CHOOSE) {
            const int j = j0 + static_cast<int>(threadIdx.x);
            count(j < size ? read(j) : 0u, j);
        }
        if (g.cluster > 1) {
            // a load from another CTA takes 1000 cycles: each CTA's bins are fetched by a warp of their own
            cluster_sync();
            if (warp < g.cluster) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float4 x = ld_cluster_f32x4(cluster_map(smem_u32(&hist[round][8 * lane + 4 * half]), warp));
                    *reinterpret_cast<float4*>(&all[warp][8 * lane + 4 * half]) = x;
                }
            }
        }
        __syncthreads();
        // the bin that holds the need-th largest: a lane has 8 bins, the first one those at the top
        if (warp == 0) {
            constexpr int EACH = BINS / 32;
            uint32_t c[EACH] = {};
            for (int r = 0; r < g.cluster; ++r) {
                const uint32_t* bins = g.cluster > 1 ? all[r] : hist[round];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint4 x = *reinterpret_cast<const uint4*>(bins + BINS - EACH * (lane + 1) + 4 * half);
                    c[4 * half] += x.x, c[4 * half + 1] += x.y, c[4 * half + 2] += x.z, c[4 * half + 3] += x.w;
                }
            }
            uint32_t sum = 0;
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                sum += c[i];
            uint32_t before = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, before, d);
                before += lane >= d ? v : 0;
            }
            before -= sum;
#pragma unroll
            for (int i = EACH - 1; i >= 0; --i) {
                if (before < need && need <= before + c[i])
                    found[round] = make_uint2(BINS - EACH * (lane + 1) + i, before);
                before += c[i];
            }
        }
        __syncthreads();
        prefix |= found[round].x << shift;
        known |= static_cast<uint32_t>(BINS - 1) << shift;
        need -= found[round].y;
    }

    // `need` of the tokens that equal T = prefix stay (none where nobody competes)
    const bool compete = g.keep > g.first + g.last;
    // each warp looks at a part of the tokens, eight a lane: the low bits tell which of them are above T
    // (or stay anyhow), the high ones which equal it
    constexpr int EACH = 8, STEP = 32 * EACH;
    const int part = ((size + WARPS - 1) / WARPS + EACH - 1) / EACH * EACH;
    const int j0 = min(warp * part, size), j1 = min(j0 + part, size);
    auto look = [&](int j) {
        uint32_t k[EACH];
        if (j + EACH <= g.held) {
#pragma unroll
            for (int i = 0; i < EACH; i += 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(keys + j + i);
                k[i] = v.x, k[i + 1] = v.y, k[i + 2] = v.z, k[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                k[i] = j + i < j1 ? key(j + i) : 0u;
        }
        uint32_t m = 0;
        if (compete && j + EACH <= j1 && lo + j >= from && lo + j + EACH <= to) {
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                m |= (k[i] > prefix ? 1u << i : 0u) | (k[i] == prefix ? 1u << (EACH + i) : 0u);
            return m;
        }
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int at = lo + j + i;
            const bool mine = j + i < j1, free = at >= from && at < to;
            m |= mine && (!free || (compete && k[i] > prefix)) ? 1u << i : 0u;
            m |= mine && free && compete && k[i] == prefix ? 1u << (EACH + i) : 0u;
        }
        return m;
    };
    constexpr uint32_t ABOVE = (1u << EACH) - 1, EQUAL = ABOVE << EACH;
    uint2 sum = make_uint2(0, 0);
    for (int j = j0; j < j1; j += STEP) {
        const uint32_t m = look(j + EACH * lane);
        sum.x += __popc(m & ABOVE);
        sum.y += __popc(m & EQUAL);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        sum.x += __shfl_xor_sync(0xffffffffu, sum.x, d);
        sum.y += __shfl_xor_sync(0xffffffffu, sum.y, d);
    }
    if (lane == 0)
        counts[warp] = sum;
    __syncthreads();
    uint2 before = make_uint2(0, 0);
    for (int w = 0; w < WARPS; ++w) {
        if (w == warp)
            sum = before;
        before.x += counts[w].x;
        before.y += counts[w].y;
    }
    if (g.cluster > 1) {
        if (threadIdx.x == 0)
            mine = before;
        cluster_sync();
        const uint32_t at = smem_u32(&mine);
        for (int r = 0; r < rank; ++r) {
            sum.x += ld_cluster_u32(cluster_map(at, r));
            sum.y += ld_cluster_u32(cluster_map(at + 4, r));
        }
    }
    for (int j = j0; j < j1; j += STEP) {
        const uint32_t m = look(j + EACH * lane), own = __popc(m & ABOVE) | __popc(m & EQUAL) << 16;
        uint32_t to_here = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, to_here, d);
            to_here += lane >= d ? v : 0;
        }
        uint32_t na = sum.x + ((to_here - own) & 0xffffu), ne = sum.y + ((to_here - own) >> 16);
        if (own) {
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                const bool a = m >> i & 1u, e = m >> (EACH + i) & 1u;
                if (a || (e && ne < need))
                    kept[na + min(ne, need)] = lo + j + EACH * lane + i;
                na += a;
                ne += e;
            }
        }
        const uint32_t last = __shfl_sync(0xffffffffu, to_here, 31);
        sum.x += last & 0xffffu;
        sum.y += last >> 16;
    }
    if (g.cluster > 1)
        cluster_sync();   // the others have read this CTA's counts
}

// A CTA takes every parts-th new page of one sequence's kv head.  A page's tokens are looked up
// (kept, page table: two dependent loads, and the weight behind them) while the one before is moved.
template <int D>
__global__ void __launch_bounds__(2 * D, 1024 / D) kv_move_kernel(const EvictArgs g)
{
    using P = Piece<D>;
    struct Source {
        const uint8_t* from[KV_PAGE];   // pieces of the tokens, null: none
        uint8_t slot[KV_PAGE];
    };
    __shared__ Source sources[2];
    grid_dep_wait();
    const int new_pages = (g.keep + KV_PAGE - 1) / KV_PAGE;
    const int part = blockIdx.x % g.parts, unit = blockIdx.x / g.parts;
    const int head = unit % g.c.kv_heads, b = unit / g.c.kv_heads;
    const int tid = threadIdx.x;
    const int stay = min(min(max(g.c.length[b], 0), g.c.max_pages * KV_PAGE), g.keep);
    if (part == 0 && head == 0 && tid == 0)
        g.new_length[b] = stay;   // may be length[b] itself: of the new value the others make the same
    const int* kept = g.kept + static_cast<size_t>(unit) * g.keep;
    const int* table = g.c.table + static_cast<size_t>(b) * g.c.max_pages;
    const int* new_table = g.new_table + static_cast<size_t>(b) * g.new_pages;
    auto old_of = [&](int page) {
        const int i = page * KV_PAGE + tid;
        return tid < KV_PAGE && page < new_pages && i < stay ? kept[i] : -1;
    };
    auto page_of = [&](int old) { return old >= 0 ? table[old / KV_PAGE] : -1; };
    auto to_of = [&](int page) { return page * KV_PAGE < stay ? new_table[page] : -1; };
    // piece of the page of token `old`; its weight
    auto tell = [&](Source& s, int old, int page, float& weight) {
        if (tid >= KV_PAGE)
            return;
        const bool held = page >= 0 && page < g.c.num_pages;
        const size_t piece = static_cast<size_t>(held ? page : 0) * g.c.kv_heads + head;
        s.from[tid] = held ? g.c.pages + piece * P::BYTES : nullptr;
        s.slot[tid] = static_cast<uint8_t>(old % KV_PAGE);
        weight = held ? g.weights[piece * KV_PAGE + old % KV_PAGE] : 0.0f;
        if (old >= 0 && !held)
            *g.c.bad = 1u;
    };
    int page = part, old = old_of(page), old1 = old_of(page + g.parts), to = to_of(page);
    float weight = 0.0f, weight1 = 0.0f;
    tell(sources[0], old, page_of(old), weight);
    __syncthreads();
    for (int turn = 0; page * KV_PAGE < stay; ++turn, page += g.parts) {
        const Source& s = sources[turn % 2];
        // on their way for the next page, and the one after it
        const int id1 = page_of(old1), old2 = old_of(page + 2 * g.parts), to1 = to_of(page + g.parts);
        const int count = min(stay - page * KV_PAGE, KV_PAGE);
        const bool there = to >= 0 && to < g.c.num_pages;
        if (there) {
            const size_t piece = static_cast<size_t>(to) * g.c.kv_heads + head;
            uint8_t* dst = g.c.pages + piece * P::BYTES;
            const uint4 none = make_uint4(0, 0, 0, 0);
            // a key's group
            const int t = tid / P::NG, gr = tid % P::NG;
            const uint8_t* f = t < count ? s.from[t] : nullptr;
            const uint4 key = f ? *reinterpret_cast<const uint4*>(f + P::k_chunk(s.slot[t], gr)) : none;
            // 16 values of two tokens
            const int p = tid / (D / 16), a = tid % (D / 16);
            const int s0 = s.slot[2 * p], s1 = s.slot[2 * p + 1];
            const uint8_t* f0 = 2 * p < count ? s.from[2 * p] : nullptr;
            const uint8_t* f1 = 2 * p + 1 < count ? s.from[2 * p + 1] : nullptr;
            const uint4 x = f0 ? *reinterpret_cast<const uint4*>(f0 + P::v_chunk(s0 / 2, a)) : none;
            const uint4 y = f1 ? *reinterpret_cast<const uint4*>(f1 + P::v_chunk(s1 / 2, a)) : none;
            // the pair's scales, one word of the two tokens' per group, and a key's scales
            const bool scales = a % 2 == 0;
            uint32_t sx = 0, sy = 0;
            if (scales) {
                sx = f0 ? *reinterpret_cast<const uint32_t*>(f0 + P::v_scale(s0 / 2, a / 2)) : 0u;
                sy = f1 ? *reinterpret_cast<const uint32_t*>(f1 + P::v_scale(s1 / 2, a / 2)) : 0u;
            }
            using W = typename std::conditional<D == 128, uint2, uint32_t>::type;
            W ks = {};
            if (tid < count && s.from[tid])
                ks = *reinterpret_cast<const W*>(s.from[tid] + P::k_scale(s.slot[tid], 0));

            const uint32_t pick = (s0 & 1 ? 0x32u : 0x10u) | (s1 & 1 ? 0x7600u : 0x5400u);
            const uint32_t z[4] = {__byte_perm(x.x, y.x, pick), __byte_perm(x.y, y.y, pick), __byte_perm(x.z, y.z, pick),
                                   __byte_perm(x.w, y.w, pick)};
            const uint32_t sz = __byte_perm(sx, sy, pick);
            if (t < count)
                *reinterpret_cast<uint4*>(dst + P::k_chunk(t, gr)) = key;
            uint8_t* at = dst + P::v_chunk(p, a);
            if (2 * p + 1 < count) {
                *reinterpret_cast<uint4*>(at) = make_uint4(z[0], z[1], z[2], z[3]);
                if (scales)
                    *reinterpret_cast<uint32_t*>(dst + P::v_scale(p, a / 2)) = sz;
            } else if (2 * p < count) {   // the other token's halves stay as they are
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    *reinterpret_cast<uint16_t*>(at + 4 * u) = static_cast<uint16_t>(z[u]);
                if (scales)
                    *reinterpret_cast<uint16_t*>(dst + P::v_scale(p, a / 2)) = static_cast<uint16_t>(sz);
            }
            if (tid < count) {
                *reinterpret_cast<W*>(dst + P::k_scale(tid, 0)) = ks;
                g.weights[piece * KV_PAGE + tid] = weight;
            }
        } else if (tid == 0) {
            *g.c.bad = 1u;
        }
        tell(sources[(turn + 1) % 2], old1, id1, weight1);
        __syncthreads();
        old1 = old2;
        to = to1;
        weight = weight1;
    }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& args, int dim, int max_kv, cudaStream_t s)
{
    EvictArgs a = args;
    const long long room = static_cast<long long>(a.c.max_pages) * KV_PAGE;
    const long long most = max_kv < room ? max_kv : room;
    const long long units = static_cast<long long>(a.c.batch) * a.c.kv_heads;
    // A cluster from 8192 tokens on while the chip is not full, whose CTAs keep 4096.  Measured, us, one
    // sequence of 8 kv heads, one CTA / clusters of 4096 tokens a CTA / of 8192: 5000 tokens 12.4 / 14.0 / -,
    // 8000 13.6 / 14.8 / -, 12000 - / 15.7 / 16.5, 30000 - / 18.7 / 20.0; 131071 472 / 37 / -.
    a.cluster = 1;
    while (most > 8192 && a.cluster < KV_MAX_CLUSTER && units * a.cluster * 2 <= 2 * 152 && most > 4096ll * a.cluster)
        a.cluster *= 2;
    constexpr int MOST = 48 * 1024;   // tokens in shared memory: what one CTA an SM has room for; others are read again
    const long long share = (most / KV_PAGE / a.cluster + 2) * KV_PAGE;
    a.held = static_cast<int>(share < MOST ? share : MOST);
    // Few tokens a CTA, or more CTAs than the chip holds: 8 warps, else 16.  8 / 16 warps, us: 2000 tokens 8.5 /
    // 9.8, 5000 12.6 / 12.4, 8000 15.3 / 13.7, 30000 by 8 CTAs 18.0 / 18.7, 131071 43.2 / 37.5; 64
    // sequences of up to 8192 144.3 / 146.3.
    const bool small = share <= 4096 + 2 * KV_PAGE || units > 2 * 152;
    static std::atomic<uint64_t> done[2];
    const auto choose = small ? kv_choose_kernel<8> : kv_choose_kernel<16>;
    cudaError_t e = kv_allow_smem(choose, MOST * 4, &done[small]);
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
    cfg.gridDim = dim3(static_cast<unsigned int>(units * a.cluster));
    cfg.blockDim = dim3(small ? 256 : 512);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.held) * 4;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    count_launch();
    if ((e = cudaLaunchKernelEx(&cfg, choose, a)) != cudaSuccess)
        return e;
    // The chip's CTAs, or more of 4 pages each for sequences of uneven length: 64 of 2000 to 8192 tokens
    // 122 us, with 8 pages 125, with the chip's alone 129, with a CTA for every page 133.
    const long long pages = (a.keep + KV_PAGE - 1) / KV_PAGE, fill = 152 * (dim == 128 ? 8 : 16) / units;
    const long long parts = fill > pages / 4 ? fill : pages / 4;
    a.parts = static_cast<int>(parts < 1 ? 1 : parts < pages ? parts : pages);
    const dim3 grid(static_cast<unsigned int>(units * a.parts));
    count_launch();
    return dim == 128 ? launch_dependent(kv_move_kernel<128>, grid, dim3(256), s, a)
                      : launch_dependent(kv_move_kernel<64>, grid, dim3(128), s, a);
}

}  // namespace mmq
