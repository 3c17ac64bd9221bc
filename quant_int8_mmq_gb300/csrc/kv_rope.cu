// kv_rope.cu -- rotary positions: of rows, and of queries and keys on their way into the
// 4-bit cache.
//
//   (a, b) -> (a cos - b sin, a sin + b cos),  angle = position * f_i of pair i (rope.cuh)
//
// Both kernels move bytes; what they compute is little beside that as long as an angle, some
// 90 instructions, is computed once for all heads of its token: a CTA fills a table of its
// tokens' cosines and sines in shared memory while its first rows are on their way, and then
// walks over the rows.  On GB300: 3314 tokens of 32 heads of 128, f32, 20 us, 5.4 TB/s (0.80 of a plain
// copy's rate), 8191 of 16 heads of 80 of which 32 turn, f16, 8.8 us, 4.8 TB/s; 64 tokens 2.2 us, a
// launch.  Into the cache 10000 tokens of 32 heads on 8 of 128: f32 69 us, 6.1 TB/s; f16 54 us, 4.0 TB/s,
// bound by issue slots (the rotation and the codes of a key, its values' and the halves of words that
// they are written in): queries alone take 31 us, keys and values 30, and 17 unturned.
#include "kv_rows.cuh"
#include "rope.cuh"

namespace mmq {
namespace {

constexpr int THREADS = 256;

// ------------------------------------------------------------------ rows
// A thread takes V pairs of a row (16 bytes of first and 16 of second values, or 32 of the pairs
// themselves), which is all that a pair needs, so rows may be turned in place; where there are
// values that stay, further threads of the row copy 2 V of them each.
template <typename T>
struct Pairs {
    static constexpr int V = 16 / static_cast<int>(sizeof(T));
    alignas(16) T a[V];
    alignas(16) T b[V];
};
constexpr int BATCH = 2;          // rows of a thread on their way at once
constexpr int TABLE = 2048;       // angles of a CTA's tokens, at most

// a: na values from x on, b: nb values from x + apart on.  `wide`: all V or none, aligned to 16 bytes.
template <typename T>
__device__ __forceinline__ void load_pairs(Pairs<T>& p, const T* x, bool wide, int na, int nb, int apart)
{
    if (wide) {
        if (na > 0)
            *reinterpret_cast<uint4*>(p.a) = *reinterpret_cast<const uint4*>(x);
        if (nb > 0)
            *reinterpret_cast<uint4*>(p.b) = *reinterpret_cast<const uint4*>(x + apart);
        return;
    }
#pragma unroll
    for (int i = 0; i < Pairs<T>::V; ++i) {
        if (i < na)
            p.a[i] = x[i];
        if (i < nb)
            p.b[i] = x[i + apart];
    }
}
template <typename T>
__device__ __forceinline__ void store_pairs(const Pairs<T>& p, T* x, bool wide, int na, int nb, int apart)
{
    if (wide) {
        if (na > 0)
            *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(p.a);
        if (nb > 0)
            *reinterpret_cast<uint4*>(x + apart) = *reinterpret_cast<const uint4*>(p.b);
        return;
    }
#pragma unroll
    for (int i = 0; i < Pairs<T>::V; ++i) {
        if (i < na)
            x[i] = p.a[i];
        if (i < nb)
            x[i + apart] = p.b[i];
    }
}

struct RopeArgs {
    KvRows x, out;
    const int* pos;
    RopeView r;
    int heads, dim, ntok;
    unsigned int heads_inv;   // 2^32 / heads, rounded up
    int toks;                 // tokens of a CTA
    int chunks, copies;       // threads of a row that turn pairs, and that copy what stays
    bool wide;
    int ctas() const { return (ntok + toks - 1) / toks; }
};

template <typename T, bool INTERLEAVED>
__device__ __forceinline__ void rope_rows(const RopeArgs& g, int cta, float2* table)
{
    constexpr int V = Pairs<T>::V;
    const int half = g.r.rot / 2, first = cta * g.toks, toks = min(g.toks, g.ntok - first);

    // the thread's chunk, the same in all its rows: `row`, `row` + step, ... of the CTA's
    const int width = g.chunks + g.copies, step = THREADS / width, chunk = threadIdx.x % width;
    const int nrow = toks * g.heads;
    int row = threadIdx.x / width;
    if (row >= step)
        row = nrow;   // more threads than rows at once
    const bool turns = chunk < g.chunks;
    int at, na, nb, apart = V;
    if (!turns) {
        at = g.r.rot + 2 * V * (chunk - g.chunks);
        na = min(V, g.dim - at);
        nb = max(0, min(V, g.dim - at - V));
    } else if (INTERLEAVED) {   // 2 V values, a then b
        at = 2 * V * chunk;
        na = min(V, g.r.rot - at);
        nb = max(0, min(V, g.r.rot - at - V));
    } else {
        at = V * chunk;
        na = nb = min(V, half - at);
        apart = half;
    }
    // token of row i; i heads < 2^32
    auto token = [&](int i) { return g.heads == 1 ? i : static_cast<int>(__umulhi(static_cast<unsigned int>(i), g.heads_inv)); };
    auto where = [&](const KvRows& r, int i) {
        const int t = token(i);
        return static_cast<T*>(r.data) + (first + t) * r.tok + (i - t * g.heads) * r.head + at;
    };
    Pairs<T> p[BATCH];
    auto load = [&](int i) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (i + k * step < nrow)
                load_pairs<T>(p[k], where(g.x, i + k * step), g.wide, na, nb, apart);
    };
    load(row);
    for (int i = threadIdx.x; i < toks * half; i += THREADS) {
        const int t = i / half;
        table[i] = rope_turn(g.r, i - t * half, g.pos[first + t]);
    }
    __syncthreads();
    for (; row < nrow; row += BATCH * step) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = row + k * step;
            if (i >= nrow)
                break;
            if (turns) {
                const float2* cs = table + token(i) * half + V * chunk;
                if constexpr (INTERLEAVED) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        T* pair = 2 * j < V ? p[k].a + 2 * j : p[k].b + (2 * j - V);
                        if (2 * j < V ? 2 * j < na : 2 * j - V < nb) {
                            const float a = Elt<T>::to(pair[0]), b = Elt<T>::to(pair[1]);
                            pair[0] = Elt<T>::from(rope_first(a, b, cs[j]));
                            pair[1] = Elt<T>::from(rope_second(a, b, cs[j]));
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (j < na) {
                            const float a = Elt<T>::to(p[k].a[j]), b = Elt<T>::to(p[k].b[j]);
                            p[k].a[j] = Elt<T>::from(rope_first(a, b, cs[j]));
                            p[k].b[j] = Elt<T>::from(rope_second(a, b, cs[j]));
                        }
                }
            }
            store_pairs<T>(p[k], where(g.out, i), g.wide, na, nb, apart);
        }
        load(row + BATCH * step);
    }
}

// Two rows a thread, five CTAs an SM: 8191 f16 rows of 16 heads of 80 8.8 us, one row 9.2, four 13.8 (spills).
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS, 5) rope_kernel(const RopeArgs g)
{
    __shared__ __align__(16) float2 table[TABLE];
    grid_dep_wait();
    grid_dep_launch();
    rope_rows<T, INTERLEAVED>(g, blockIdx.x, table);
}

template <typename T>
RopeArgs rope_args(const KvRows& x, const KvRows& out, const int* pos, const RopeView& r, int heads, int dim, int ntok, bool wide)
{
    constexpr int V = Pairs<T>::V;
    const int half = r.rot / 2;
    RopeArgs a = {x, out, pos, r, heads, dim, ntok, 0, 1, (half + V - 1) / V, 0, wide && half % V == 0 && dim % V == 0};
    if (x.data != out.data || x.tok != out.tok || x.head != out.head)   // in place nothing is copied
        a.copies = (dim - r.rot + 2 * V - 1) / (2 * V);
    a.heads_inv = static_cast<unsigned int>(((1ull << 32) + heads - 1) / heads);
    // tokens of a CTA: up to four rows a thread while the chip stays full, one at least (8191 tokens of
    // 16 heads of 80, f16, four rows 8.9 us, one 10.9; 64 tokens of 32 heads 2.2 with one)
    const int step = THREADS / (a.chunks + a.copies);
    for (int rows = 4; rows >= 1; rows /= 2) {
        a.toks = rows * step / heads;
        a.toks = a.toks < TABLE / half ? a.toks : TABLE / half;
        a.toks = a.toks < 1 ? 1 : a.toks;
        if (a.ctas() >= 152 * 6)
            break;
    }
    return a;
}

// ------------------------------------------------------------------ into the cache
// The first CTAs have keys and values, the others queries, which are rows as above.  A lane has 8
// values of a key or value, D / 8 lanes a row, 2 rows of 128 values (4 of 64) a warp at once; one pass's
// rows are loaded while the last one's are turned.
constexpr int WARPS = THREADS / 32;

// Where a value's partner is.  HALVES: a lane has four values of one half of what turns and the four
// they pair with (and, of what stays, four of each half), which takes 32-value groups to lie in
// one or the other.  INSIDE: 8 consecutive values, pairs among them.  ANYWHERE: 8 consecutive values,
// partners read from memory.
enum RopePairs { HALVES = 0, INSIDE = 1, ANYWHERE = 2 };

struct EnterArgs {
    KvView c;
    KvRows k, v;
    RopeArgs q;            // and positions, the plan and the number of tokens
    int toks;              // tokens of a CTA of keys and values: 1, 2, 4 or 8
    int ctas;              // of keys and values: the longer ones, and the first
    bool wide;             // keys and values
};

// The two fours of values of lane l: from first and from second on (8 consecutive ones in the other
// layouts).
struct Fours {
    int first, second;
    bool turns;
    int pair;              // of the first value
};
template <int PAIRS>
__device__ __forceinline__ Fours fours_of(int l, int dim, int rot)
{
    if constexpr (PAIRS != HALVES)
        return {8 * l, 8 * l + 4, true, 0};
    const int half = rot / 2, stay = dim - rot;
    return 4 * l < half ? Fours{4 * l, half + 4 * l, true, 4 * l}
                        : Fours{half + 4 * l, half + 4 * l + stay / 2, false, 0};
}
template <typename T>
__device__ __forceinline__ void load_fours(const T* row, const Fours& f, bool wide, float (&x)[8])
{
    const float4 a = load4(row + f.first, wide), b = load4(row + f.second, wide);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

template <int PAIRS, typename T>
__device__ __forceinline__ void turn8(float (&x)[8], const T* row, int l, const Fours& f, const RopeView& r, const float2* cs)
{
    const int half = r.rot / 2;
    if constexpr (PAIRS == HALVES) {
        if (f.turns) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 c = cs[f.pair + j];
                const float a = x[j], b = x[4 + j];
                x[j] = rope_first(a, b, c);
                x[4 + j] = rope_second(a, b, c);
            }
        }
    } else if constexpr (PAIRS == INSIDE) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * l + j < half) {
                const float2 c = cs[4 * l + j];
                const float a = x[2 * j], b = x[2 * j + 1];
                x[2 * j] = rope_first(a, b, c);
                x[2 * j + 1] = rope_second(a, b, c);
            }
    } else {
        row += 8 * l;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int d = 8 * l + j;
            if (d < r.rot) {
                const bool lower = d < half;
                const float y = Elt<T>::to(row[lower ? half : -half]);
                const float2 c = cs[lower ? d : d - half];
                x[j] = lower ? rope_first(x[j], y, c) : rope_second(y, x[j], c);
            }
            ++row;
        }
    }
}

// A key row whose lanes have two fours each: the largest of a group among 8 lanes, and words of
// codes put together by two lanes, the even one of its first group's, the odd one of its second's.
template <int D>
__device__ __forceinline__ void put_key_fours(const float (&x)[8], const Fours& f, int l, int slot, uint8_t* piece, bool store)
{
    using P = Piece<D>;
    uint32_t word[2];
    float s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float y[4], a = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[i] = x[4 * h + i] == x[4 * h + i] ? x[4 * h + i] : 0.0f;   // no number is 0
            a = fmaxf(a, fabsf(y[i]));
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1)
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
        s[h] = kv_scale(a);
        uint32_t n[4];
        kv_codes(y, s[h], n);
        word[h] = (n[0] & 15u) | (n[2] & 15u) << 4 | (n[1] & 15u) << 16 | (n[3] & 15u) << 20;
    }
    const bool odd = l & 1;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? word[0] : word[1], 1);
    const uint32_t own = odd ? other | word[1] << 8 : word[0] | other << 8;
    const int from = odd ? f.second : f.first, group = from / 32;
    if (!store)
        return;
    *reinterpret_cast<uint32_t*>(piece + P::k_chunk(slot, group) + from % 32 / 8 * 4) = own;
    if (l % 8 < 2)
        *reinterpret_cast<__half*>(piece + P::k_scale(slot, group)) = __float2half_rn(odd ? s[1] : s[0]);   // exact
}

// Five CTAs an SM: 10000 f16 tokens of 32 heads on 8 54 us, with four 57, with six (28 bytes spilled) and one
// row a thread 52, but 2500 of 8 on one of 64 values 7.4 for 6.5.
template <int D, typename T, int PAIRS>
__global__ void __launch_bounds__(THREADS, 5) kv_write_rope_kernel(const EnterArgs g)
{
    using P = Piece<D>;
    constexpr int LANES = D / 8, AT_ONCE = 32 / LANES;
    __shared__ __align__(16) float2 table[TABLE];
    static_assert(WARPS * D / 2 <= TABLE, "table");
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    grid_dep_wait();
    grid_dep_launch();
    if (static_cast<int>(blockIdx.x) >= g.ctas)
        return rope_rows<T, PAIRS == INSIDE>(g.q, blockIdx.x - g.ctas, table);
    const RopeView& r = g.q.r;
    const int half = r.rot / 2, first = blockIdx.x * g.toks, toks = min(g.toks, g.q.ntok - first);

    const int warps = WARPS / g.toks;                    // of a token
    const int tok = min(warp / warps, toks - 1);         // a last CTA's spare warps compute and store nothing
    const bool spare = warp / warps >= toks;
    const int t = first + tok, hk = g.c.kv_heads;
    const int l = lane % LANES, sub = warp % warps * AT_ONCE + lane / LANES, step = warps * AT_ONCE;
    const Fours mine = fours_of<PAIRS>(l, D, r.rot), plain = {8 * l, 8 * l + 4, false, 0};
    // passes over the rows: keys, values
    const int each = (hk + step - 1) / step, passes = 2 * each;
    auto row_of = [&](int pass) -> const T* {
        const KvRows& in = pass < each ? g.k : g.v;
        const int h = min((pass < each ? pass : pass - each) * step + sub, hk - 1);
        return static_cast<const T*>(in.data) + t * in.tok + h * in.head;
    };
    const T* row = row_of(0);
    float ahead[8];
    load_fours(row, mine, g.wide, ahead);
    for (int i = threadIdx.x; i < toks * half; i += THREADS)
        table[i] = rope_turn(r, i % half, g.q.pos[first + i / half]);
    int slot;
    const long long page = kv_page_of(g.c, t, static_cast<long long>(hk) * P::BYTES, lane, &slot);
    const float2* cs = table + tok * half;
    __syncthreads();

    for (int pass = 0; pass < passes; ++pass) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = ahead[j];
        const T* here = row;
        if (pass + 1 < passes) {
            row = row_of(pass + 1);
            load_fours(row, pass + 1 >= each ? plain : mine, g.wide, ahead);
        }
        const int h = (pass < each ? pass : pass - each) * step + sub;
        const bool store = h < hk && page >= 0 && !spare;
        uint8_t* piece = g.c.pages + page + h * P::BYTES;
        if (pass < each) {
            turn8<PAIRS>(x, here, l, mine, r, cs);
            if constexpr (PAIRS == HALVES) {
                put_key_fours<D>(x, mine, l, slot, piece, store);
            } else {
                const Codes8 codes = kv_quantise8(x, true);
                if (store)
                    Place8<D>(slot, l, true).put(piece, codes, l, true);
            }
        } else {
            const Codes8 codes = kv_quantise8(x, false);
            if (store)
                Place8<D>(slot, l, false).put(piece, codes, l, false);
        }
    }
}

template <int D, typename T>
cudaError_t launch_enter(EnterArgs a, const KvRows& q, const KvRows& q_out, const int* pos, const RopeView& r, int heads, int ntok,
                         bool wide_q, cudaStream_t s)
{
    a.q = rope_args<T>(q, q_out, pos, r, heads, D, ntok, wide_q);
    // More tokens a CTA fill its warps with few heads and share the wait for the first rows; fewer end
    // together.  A CTA's time goes with its passes.  Measured, us, 1 / 2 / 4 / 8 tokens: 700 tokens of 8 kv
    // heads 8.0 / 6.2 / 5.9 / 9.0 (f16, 128 values), of 32 10.6 / 13.0 / 14.9 / 26.3; 10000 tokens of 8
    // 92 / 65 / 59 / 57, of 32 136 / 126 / 120 / 117, of one of 64 values 56 / 31 / 19 / 13 (four CTAs an SM).
    for (a.toks = 8; a.toks > 1; a.toks /= 2) {
        const int at_once = WARPS / a.toks * (256 / D);
        if (3ll * ((ntok + a.toks - 1) / a.toks) >= 2ll * 152 * ((a.c.kv_heads + at_once - 1) / at_once))
            break;
    }
    a.ctas = (ntok + a.toks - 1) / a.toks;
    const dim3 grid(static_cast<unsigned int>(a.ctas + a.q.ctas())), block(THREADS);
    count_launch();
    if (r.interleaved)
        return launch_dependent(kv_write_rope_kernel<D, T, INSIDE>, grid, block, s, a);
    // the partners that come with a lane's own values, 62 us, and those read from memory, 103 (3 prompts of
    // up to 3314 tokens, 32 heads on 8 of 128, f32, with the cache read back)
    if (r.rot % 64 == 0 && (D - r.rot) % 64 == 0)
        return launch_dependent(kv_write_rope_kernel<D, T, HALVES>, grid, block, s, a);
    return launch_dependent(kv_write_rope_kernel<D, T, ANYWHERE>, grid, block, s, a);
}

template <typename T>
cudaError_t launch_rows(const KvRows& x, const KvRows& out, const int* pos, const RopeView& r, int heads, int dim, int ntok,
                        bool wide, cudaStream_t s)
{
    const RopeArgs a = rope_args<T>(x, out, pos, r, heads, dim, ntok, wide);
    count_launch();
    return launch_dependent(r.interleaved ? rope_kernel<T, true> : rope_kernel<T, false>, dim3(static_cast<unsigned int>(a.ctas())),
                            dim3(THREADS), s, a);
}

}  // namespace

cudaError_t launch_rope(const KvRows& x, const KvRows& out, const int* pos, const RopeView& r, int dtype, int heads,
                        int dim, int ntok, bool wide, cudaStream_t s)
{
    const auto launch = dtype == KV_F32 ? launch_rows<float> : dtype == KV_F16 ? launch_rows<__half> : launch_rows<__nv_bfloat16>;
    return launch(x, out, pos, r, heads, dim, ntok, wide, s);
}

cudaError_t launch_kv_write_rope(const KvView& c, int dim, int dtype, const KvRows& q, const KvRows& q_out, int heads,
                                 const KvRows& k, const KvRows& v, const int* pos, const RopeView& r, bool wide_q,
                                 bool wide_kv, int ntok, cudaStream_t s)
{
    EnterArgs a = {};
    a.c = c;
    a.k = k;
    a.v = v;
    a.wide = wide_kv;
    const auto launch = dim == 128 ? (dtype == KV_F32   ? launch_enter<128, float>
                                      : dtype == KV_F16 ? launch_enter<128, __half>
                                                        : launch_enter<128, __nv_bfloat16>)
                                   : (dtype == KV_F32   ? launch_enter<64, float>
                                      : dtype == KV_F16 ? launch_enter<64, __half>
                                                        : launch_enter<64, __nv_bfloat16>);
    return launch(a, q, q_out, pos, r, heads, ntok, wide_q, s);
}

}  // namespace mmq
