// kv_rope.cu -- rotary positions: of rows, and of queries and keys on their way into the
// 4-bit cache.
//
//   (a, b) -> (a cos - b sin, a sin + b cos),  angle = position * f_i of pair i (rope.cuh)
//
// Both kernels move bytes; what they compute is little beside that as long as an angle, some
// 90 instructions, is computed once for all heads of its token: a CTA fills a table of its
// tokens' cosines and sines in shared memory while its first rows are on their way, and then
// walks over the rows.
#include "kv_rows.cuh"
#include "rope.cuh"

namespace mmq {
namespace {

constexpr int THREADS = 256;

// ------------------------------------------------------------------ rows
// A thread takes V pairs of a row (16 bytes of first and 16 of second values, or of the pairs
// themselves), which is all that a pair needs, so rows may be turned in place; where there are
// values that stay, further threads of the row copy 2 V of them each.
template <typename T>
struct Pairs {
    static constexpr int V = 16 / static_cast<int>(sizeof(T));
    alignas(16) T a[V];
    alignas(16) T b[V];
};
constexpr int BATCH = 4;          // rows of a thread on their way at once
constexpr int TABLE = 2048;       // angles of a CTA's tokens, at most

// `wide`: every chunk is whole and aligned to 16 bytes.  Else element by element: na and nb
// of a and b, the b's `apart` after the a's, elements of a `step` apart.
template <typename T>
__device__ __forceinline__ void load_pairs(Pairs<T>& p, const T* x, bool wide, int na, int nb, int step, int apart)
{
    constexpr int V = Pairs<T>::V;
    if (wide) {
        const int second = step == 1 ? apart : V;
        if (na > 0)
            *reinterpret_cast<uint4*>(p.a) = *reinterpret_cast<const uint4*>(x);
        if (nb > 0)
            *reinterpret_cast<uint4*>(p.b) = *reinterpret_cast<const uint4*>(x + second);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i < na)
            p.a[i] = x[i * step];
        if (i < nb)
            p.b[i] = x[i * step + apart];
    }
}
template <typename T>
__device__ __forceinline__ void store_pairs(const Pairs<T>& p, T* x, bool wide, int na, int nb, int step, int apart)
{
    constexpr int V = Pairs<T>::V;
    if (wide) {
        const int second = step == 1 ? apart : V;
        if (na > 0)
            *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(p.a);
        if (nb > 0)
            *reinterpret_cast<uint4*>(x + second) = *reinterpret_cast<const uint4*>(p.b);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i < na)
            x[i * step] = p.a[i];
        if (i < nb)
            x[i * step + apart] = p.b[i];
    }
}

struct RopeArgs {
    KvRows x, out;
    const int* pos;
    RopeView r;
    int heads, dim, ntok;
    int toks;              // tokens of a CTA
    int chunks, copies;    // threads of a row that turn pairs, and that copy what stays
    bool wide;
};

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rope_kernel(const RopeArgs g)
{
    constexpr int V = Pairs<T>::V;
    __shared__ float2 table[TABLE];
    const int half = g.r.rot / 2, first = blockIdx.x * g.toks, toks = min(g.toks, g.ntok - first);
    grid_dep_wait();
    grid_dep_launch();

    // the thread's chunk, the same in all its rows: rows[0], rows[0] + step, ... of the CTA's
    const int width = g.chunks + g.copies, step = THREADS / width, chunk = threadIdx.x % width;
    const int nrow = toks * g.heads;
    int row = threadIdx.x / width;
    if (row >= step)
        row = nrow;   // more threads than rows at once
    const bool turns = chunk < g.chunks;
    int at, na, nb, apart, stride;
    if (turns) {
        at = INTERLEAVED ? 2 * V * chunk : V * chunk;
        na = nb = min(V, half - V * chunk);
        apart = INTERLEAVED ? 1 : half;
        stride = INTERLEAVED ? 2 : 1;
    } else {
        at = g.r.rot + 2 * V * (chunk - g.chunks);
        na = min(V, g.dim - at);
        nb = max(0, min(V, g.dim - at - V));
        apart = V;
        stride = 1;
    }
    auto where = [&](const KvRows& r, int i) {
        return static_cast<T*>(r.data) + (first + i / g.heads) * r.tok + i % g.heads * r.head + at;
    };
    Pairs<T> p[BATCH];
    auto load = [&](int i) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (i + k * step < nrow)
                load_pairs<T>(p[k], where(g.x, i + k * step), g.wide, na, nb, stride, apart);
    };
    load(row);
    for (int i = threadIdx.x; i < toks * half; i += THREADS)
        table[i] = rope_turn(g.r, i % half, g.pos[first + i / half]);
    __syncthreads();
    for (; row < nrow; row += BATCH * step) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = row + k * step;
            if (i >= nrow)
                break;
            if (turns) {
                const float2* cs = table + i / g.heads * half + V * chunk;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (j >= na)
                        break;
                    T& u = INTERLEAVED && g.wide ? (2 * j < V ? p[k].a[2 * j % V] : p[k].b[2 * j % V]) : p[k].a[j];
                    T& v = INTERLEAVED && g.wide ? (2 * j < V ? p[k].a[2 * j % V + 1] : p[k].b[2 * j % V + 1]) : p[k].b[j];
                    const float a = Elt<T>::to(u), b = Elt<T>::to(v);
                    u = Elt<T>::from(rope_first(a, b, cs[j]));
                    v = Elt<T>::from(rope_second(a, b, cs[j]));
                }
            }
            store_pairs<T>(p[k], where(g.out, i), g.wide, na, nb, stride, apart);
        }
        load(row + BATCH * step);
    }
}

// ------------------------------------------------------------------ into the cache
// The lanes of kv_rows.cuh: 8 values a lane, D / 8 lanes a row, 2 rows of 128 values (4 of 64)
// a warp at once.  A token's keys and values come first, then its queries; one pass's rows are
// loaded while the last one's are turned.
constexpr int WARPS = THREADS / 32;

enum RopePairs { BY_LANES = 0, INSIDE = 1, ANYWHERE = 2 };   // where a value's partner is

struct EnterArgs {
    KvView c;
    KvRows q, q_out, k, v;
    const int* pos;
    RopeView r;
    int heads, ntok;
    int toks;              // tokens of a CTA: 1, 2, 4 or 8
    bool wide_q, wide_kv;
};

template <int D, int PAIRS, typename T>
__device__ __forceinline__ void turn8(float (&x)[8], const T* row, int l, const RopeView& r, const float2* cs)
{
    const int half = r.rot / 2;
    if constexpr (PAIRS == INSIDE) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * l + j < half) {
                const float2 c = cs[4 * l + j];
                const float a = x[2 * j], b = x[2 * j + 1];
                x[2 * j] = rope_first(a, b, c);
                x[2 * j + 1] = rope_second(a, b, c);
            }
    } else if constexpr (PAIRS == BY_LANES) {   // half is a multiple of 8
        const int lanes = half / 8;
        const bool lower = l < lanes, turns = l < 2 * lanes;
        const int lane = threadIdx.x % 32, from = turns ? lower ? lane + lanes : lane - lanes : lane;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = __shfl_sync(0xffffffffu, x[j], from);
        if (turns) {
            const float2* c = cs + 8 * (lower ? l : l - lanes);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = lower ? rope_first(x[j], y[j], c[j]) : rope_second(y[j], x[j], c[j]);
        }
    } else {
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

template <int D, typename T, int PAIRS>
__global__ void __launch_bounds__(THREADS) kv_write_rope_kernel(const EnterArgs g)
{
    using P = Piece<D>;
    constexpr int LANES = D / 8, AT_ONCE = 32 / LANES;
    __shared__ float2 table[WARPS * D / 2];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int half = g.r.rot / 2, first = blockIdx.x * g.toks, toks = min(g.toks, g.ntok - first);
    grid_dep_wait();
    grid_dep_launch();

    const int warps = WARPS / g.toks;                    // of a token
    const int tok = min(warp / warps, toks - 1);         // a last CTA's spare warps compute and store nothing
    const bool spare = warp / warps >= toks;
    const int t = first + tok, hk = g.c.kv_heads;
    const int l = lane % LANES, sub = warp % warps * AT_ONCE + lane / LANES, step = warps * AT_ONCE;
    // passes over the rows: keys and values, then queries
    const int enters = (2 * hk + step - 1) / step, passes = enters + (g.heads + step - 1) / step;
    auto row_of = [&](int pass) -> const T* {
        const KvRows* in;
        int h;
        if (pass < enters) {
            const int i = min(pass * step + sub, 2 * hk - 1);
            in = i < hk ? &g.k : &g.v;
            h = i < hk ? i : i - hk;
        } else {
            in = &g.q;
            h = min((pass - enters) * step + sub, g.heads - 1);
        }
        return static_cast<const T*>(in->data) + t * in->tok + h * in->head + 8 * l;
    };
    const T* row = row_of(0);
    float ahead[8];
    load8(row, g.wide_kv, ahead);
    for (int i = threadIdx.x; i < toks * half; i += THREADS)
        table[i] = rope_turn(g.r, i % half, g.pos[first + i / half]);
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
            load8(row, pass + 1 < enters ? g.wide_kv : g.wide_q, ahead);
        }
        if (pass < enters) {
            const int i = pass * step + sub;
            const bool key = i < hk;
            if (__any_sync(0xffffffffu, key)) {
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = x[j];
                turn8<D, PAIRS>(y, here, l, g.r, cs);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = key ? y[j] : x[j];
            }
            const Codes8 codes = kv_quantise8(x, key);
            if (i < 2 * hk && page >= 0 && !spare)
                Place8<D>(slot, l, key).put(g.c.pages + page + (key ? i : i - hk) * P::BYTES, codes, l, key);
        } else {
            const int h = (pass - enters) * step + sub;
            turn8<D, PAIRS>(x, here, l, g.r, cs);
            __syncwarp();   // in place: every lane has what it needs of the row
            if (h < g.heads && !spare)
                store8(static_cast<T*>(g.q_out.data) + t * g.q_out.tok + h * g.q_out.head + 8 * l, g.wide_q, x);
        }
    }
}

template <int D, typename T>
cudaError_t launch_enter(const EnterArgs& a, cudaStream_t s)
{
    const dim3 grid(static_cast<unsigned int>((a.ntok + a.toks - 1) / a.toks)), block(THREADS);
    count_launch();
    if (a.r.interleaved)
        return launch_dependent(kv_write_rope_kernel<D, T, INSIDE>, grid, block, s, a);
    if (a.r.rot % 16 == 0)
        return launch_dependent(kv_write_rope_kernel<D, T, BY_LANES>, grid, block, s, a);
    return launch_dependent(kv_write_rope_kernel<D, T, ANYWHERE>, grid, block, s, a);
}

}  // namespace

cudaError_t launch_rope(const KvRows& x, const KvRows& out, const int* pos, const RopeView& r, int dtype, int heads,
                        int dim, int ntok, bool wide, cudaStream_t s)
{
    const int v = dtype == KV_F32 ? 4 : 8, half = r.rot / 2;
    RopeArgs a = {x, out, pos, r, heads, dim, ntok, 1, (half + v - 1) / v, 0, wide && half % v == 0 && dim % v == 0};
    if (x.data != out.data || x.tok != out.tok || x.head != out.head)   // in place nothing is copied
        a.copies = (dim - r.rot + 2 * v - 1) / (2 * v);
    // tokens of a CTA: rows enough for its threads
    const int step = THREADS / (a.chunks + a.copies);
    int toks = step / heads;
    toks = toks < 1 ? 1 : toks;
    toks = toks < TABLE / half ? toks : TABLE / half;
    a.toks = toks;
    const dim3 grid(static_cast<unsigned int>((ntok + toks - 1) / toks)), block(THREADS);
    count_launch();
    auto launch = [&](auto kernel) { return launch_dependent(kernel, grid, block, s, a); };
    if (r.interleaved)
        return dtype == KV_F32   ? launch(rope_kernel<float, true>)
               : dtype == KV_F16 ? launch(rope_kernel<__half, true>)
                                 : launch(rope_kernel<__nv_bfloat16, true>);
    return dtype == KV_F32   ? launch(rope_kernel<float, false>)
           : dtype == KV_F16 ? launch(rope_kernel<__half, false>)
                             : launch(rope_kernel<__nv_bfloat16, false>);
}

cudaError_t launch_kv_write_rope(const KvView& c, int dim, int dtype, const KvRows& q, const KvRows& q_out, int heads,
                                 const KvRows& k, const KvRows& v, const int* pos, const RopeView& r, bool wide_q,
                                 bool wide_kv, int ntok, cudaStream_t s)
{
    EnterArgs a = {c, q, q_out, k, v, pos, r, heads, ntok, 1, wide_q, wide_kv};
    a.toks = ntok >= 8 * 152 * 8 ? 8 : ntok >= 4 * 152 * 8 ? 4 : ntok >= 2 * 152 * 8 ? 2 : 1;
    if (dim == 128)
        return dtype == KV_F32   ? launch_enter<128, float>(a, s)
               : dtype == KV_F16 ? launch_enter<128, __half>(a, s)
                                 : launch_enter<128, __nv_bfloat16>(a, s);
    return dtype == KV_F32   ? launch_enter<64, float>(a, s)
           : dtype == KV_F16 ? launch_enter<64, __half>(a, s)
                             : launch_enter<64, __nv_bfloat16>(a, s);
}

}  // namespace mmq
