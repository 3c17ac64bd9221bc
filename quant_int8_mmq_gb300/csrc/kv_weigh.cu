// kv_weigh.cu -- the weight that each key of the 4-bit cache receives from the new tokens' rows:
//
//   out[j] = decay in[j] (tokens that were there) + sum over rows 2^(x_j - ref) / sum,
//   x_j = scale log2(e) q . k_j
//
// with each row's reference and sum from the attention that ran before.  A warp owns a page, so
// a key's sum over the rows stays in registers and is written once, in one order.
#include "kv.cuh"

namespace mmq {
namespace {

constexpr int WARPS = 4;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Rows staged at a time, as operands of mma m16n8k16 (kv_step.cu): f32 rows as 8 of hi and 8 of
// lo parts, 16-bit rows 16 at a time.
template <int D, typename T>
struct WeighSmem {
    static constexpr bool HL = sizeof(T) == 4;
    static constexpr int ROWS = HL ? 8 : 16;      // of a tile
    static constexpr int TILES = 4;
    static constexpr int CHUNK = ROWS * TILES;    // rows staged at a time
    uint4 q[TILES][D / 16][32];
    float coef[CHUNK], ref[CHUNK], inv[CHUNK];
    int pos[CHUNK];
};

template <int D, typename T>
__global__ void __launch_bounds__(WARPS * 32) kv_weigh_kernel(const WeighArgs w)
{
    using P = Piece<D>;
    using S = WeighSmem<D, T>;
    constexpr bool HL = S::HL;
    constexpr int ROWS = S::ROWS, SETS = ROWS / 8;
    __shared__ S sm;
    const AttendArgs& g = w.a;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int n = lane / 4, t = lane % 4;
    grid_dep_wait();
    int id = blockIdx.x;
    const int part = id % w.parts;
    id /= w.parts;
    const int head = id % g.c.kv_heads, b = id / g.c.kv_heads;
    const int first = g.c.start[b], last = g.c.start[b + 1];
    if (first < 0 || last <= first || last > g.ntok)
        return;
    const int rows_b = (last - first) * g.group;
    const int length = min(max(g.c.length[b], 0), g.c.max_pages * KV_PAGE);
    const int pos0 = max(g.c.length[b], 0) - (last - first);
    const int npage = (length + KV_PAGE - 1) / KV_PAGE;
    const int* table = g.c.table + static_cast<size_t>(b) * g.c.max_pages;

    int staged = -1;   // the chunk of rows in shared memory
    for (int base = part * WARPS; base < npage; base += w.parts * WARPS) {
        const int i = base + warp, kbase = i * KV_PAGE;
        int pid = i < npage ? table[i] : -1;
        if (i < npage && (pid < 0 || pid >= g.c.num_pages)) {
            *g.c.bad = 1u;
            pid = -1;
        }
        const size_t piece = static_cast<size_t>(max(pid, 0)) * g.c.kv_heads + head;
        const uint8_t* page = g.c.pages + piece * P::BYTES;
        float acc[8][2];
#pragma unroll
        for (int o = 0; o < 8; ++o)
            acc[o][0] = acc[o][1] = 0.0f;
        // rows that see one of the CTA's four pages
        const long long from = max(static_cast<long long>(base) * KV_PAGE - pos0, 0ll) * g.group;
        long long to = rows_b;
        if (g.window > 0 && g.sinks <= base * KV_PAGE) {
            const long long seen = static_cast<long long>(base + WARPS) * KV_PAGE - 1 + g.window - pos0;   // positions below
            to = min(to, max(seen, 0ll) * g.group);
        }
        for (int chunk = static_cast<int>(from / S::CHUNK); chunk < (to + S::CHUNK - 1) / S::CHUNK; ++chunk) {
            if (chunk != staged) {
                __syncthreads();
                for (int r = warp; r < S::CHUNK; r += WARPS) {
                    const int row = chunk * S::CHUNK + r;
                    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    float2 stats = make_float2(0.0f, 0.0f);
                    if (row < rows_b) {
                        const long long token = first + row / g.group;
                        const int h = head * g.group + row % g.group;
                        stats = g.stats[token * g.heads + h];
                        if (stats.y > 0.0f && lane < D / 4)   // a row that is no number has none
                            x = load4(static_cast<const T*>(g.q.data) + token * g.q.tok + h * g.q.head + 4 * lane, g.wide);
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
                        const int step = 4 * lane % (D / 4) / 4, owner = r % 8 * 4 + 4 * lane / (D / 4);
                        uint32_t* at = reinterpret_cast<uint32_t*>(&sm.q[r / ROWS][step][owner]);
                        if constexpr (HL) {
                            *reinterpret_cast<uint4*>(at) = make_uint4(hi.x, lo.x, hi.y, lo.y);
                        } else {
                            at[r / 8 % 2] = hi.x;
                            at[2 + r / 8 % 2] = hi.y;
                        }
                    }
                    if (lane == 0) {
                        sm.coef[r] = fminf(fmaxf(g.scale_log2 * kv_pow2(e), 1e-38f), 1e38f);
                        sm.ref[r] = stats.x;
                        sm.inv[r] = stats.y;
                        sm.pos[r] = row < rows_b ? pos0 + row / g.group : -1;
                    }
                }
                __syncthreads();
                staged = chunk;
            }
            if (pid < 0)
                continue;
            const int tiles = min(S::TILES, (rows_b - chunk * S::CHUNK + ROWS - 1) / ROWS);
#pragma unroll 1
            for (int oct = 0; oct < 8; oct += 2) {
                uint32_t k[2][D / 16][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int token = 8 * (oct + h) + n;
                    uint32_t v[D / 32];
                    if constexpr (D == 128) {
                        const uint4 u = *reinterpret_cast<const uint4*>(page + P::k_chunk(token, t));
                        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2*>(page + P::k_chunk(token, t / 2) + t % 2 * 8);
                        v[0] = u.x, v[1] = u.y;
                    }
                    const __half2 s =
                        __half2half2(*reinterpret_cast<const __half*>(page + P::k_scale(token, D == 128 ? t : t / 2)));
                    const __half2 sb = kv_addend(s);
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {
                        k[h][2 * j][0] = kv_h2u(kv_widen<0>(v[j], s, sb));
                        k[h][2 * j][1] = kv_h2u(kv_widen<1>(v[j], s, sb));
                        k[h][2 * j + 1][0] = kv_h2u(kv_widen<2>(v[j], s, sb));
                        k[h][2 * j + 1][1] = kv_h2u(kv_widen<3>(v[j], s, sb));
                    }
                }
                float sum[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
                for (int tile = 0; tile < tiles; ++tile) {
                    float c[2][4] = {};
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        const uint4 q = sm.q[tile][j][lane];
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            mma16816(c[h], q.x, q.y, q.z, q.w, k[h][j][0], k[h][j][1]);
                    }
#pragma unroll
                    for (int s = 0; s < SETS; ++s) {
                        const int r = tile * ROWS + n + 8 * s;
                        const float coef = sm.coef[r], ref = sm.ref[r], inv = sm.inv[r];
                        const uint64_t seen = kv_seen_bits(sm.pos[r], kbase, g.window, g.sinks) >> (8 * oct + 2 * t);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float x = HL ? c[h][e] + c[h][e + 2] : c[h][e + 2 * s];
                                const float p = kv_ex2(fmaf(x, coef, -ref));
                                if (seen >> (8 * h + e) & 1u)
                                    sum[h][e] = fmaf(p, inv, sum[h][e]);
                            }
                    }
                }
#pragma unroll
                for (int o = 0; o < 8; ++o)
                    if (o == oct) {
                        acc[o][0] += sum[0][0], acc[o][1] += sum[0][1];
                        acc[(o + 1) % 8][0] += sum[1][0], acc[(o + 1) % 8][1] += sum[1][1];
                    }
            }
        }
        if (pid < 0)
            continue;
        // over the eight rows of a tile's lanes: each step hands half of the keys to the partner,
        // until lane (n, t) has those of octet n
#pragma unroll
        for (int half = 4; half >= 1; half /= 2) {
            const bool upper = n & half;
#pragma unroll
            for (int o = 0; o < half; ++o)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float send = upper ? acc[o][e] : acc[o + half][e];
                    const float stay = upper ? acc[o + half][e] : acc[o][e];
                    acc[o][e] = stay + __shfl_xor_sync(0xffffffffu, send, 4 * half);
                }
        }
        const int j = kbase + 8 * n + 2 * t;   // this lane's keys: j, j + 1
        const size_t at = piece * KV_PAGE + 8 * n + 2 * t;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (j + e < length)
                w.out[at + e] = (j + e < pos0 ? w.decay * w.in[at + e] : 0.0f) + acc[0][e];
    }
}

template <int D, typename T>
cudaError_t launch_weigh(const WeighArgs& a, cudaStream_t s)
{
    const long long grid = static_cast<long long>(a.a.c.batch) * a.a.c.kv_heads * a.parts;
    count_launch();
    return launch_dependent(kv_weigh_kernel<D, T>, dim3(static_cast<unsigned int>(grid)), dim3(WARPS * 32), s, a);
}

}  // namespace

cudaError_t launch_kv_weigh(const WeighArgs& args, int dim, int dtype, int max_kv, cudaStream_t s)
{
    WeighArgs a = args;
    const long long units = static_cast<long long>(a.a.c.batch) * a.a.c.kv_heads;
    long long pages = (static_cast<long long>(max_kv) + KV_PAGE - 1) / KV_PAGE;
    pages = pages < a.a.c.max_pages ? pages : a.a.c.max_pages;
    // the chip's CTAs, or parts of 32 pages where lengths are uneven, of 4 at least
    long long parts = 4 * 152 / units;
    parts = parts > pages / 32 ? parts : pages / 32;
    parts = parts < pages / 4 ? parts : pages / 4;
    parts = parts < 0x7fffffffll / units ? parts : 0x7fffffffll / units;
    a.parts = static_cast<int>(parts < 1 ? 1 : parts);
    if (dim == 128)
        return dtype == KV_F32   ? launch_weigh<128, float>(a, s)
               : dtype == KV_F16 ? launch_weigh<128, __half>(a, s)
                                 : launch_weigh<128, __nv_bfloat16>(a, s);
    return dtype == KV_F32   ? launch_weigh<64, float>(a, s)
           : dtype == KV_F16 ? launch_weigh<64, __half>(a, s)
                             : launch_weigh<64, __nv_bfloat16>(a, s);
}

}  // namespace mmq
