// kv_api.cu -- entry points of the 4-bit key/value cache, of the attention over it and the
// weights it gives, of eviction by them, and of rotary positions.
//
// As in api.cu, arguments are checked on the host before any CUDA call; what only the
// device knows (page ids, lengths) is checked by the kernels.
#include <cmath>

#include "api.h"
#include "kv.cuh"
#include "rope.cuh"

namespace mmq {

// How an attention call is cut up: rows to row tiles and, where those are few, the visible
// pages to parts.  Depends on the arguments alone (the chip has 152 SMs).
AttendPlan plan_attend(int dtype, int heads, int kv_heads, int dim, int batch, int ntok, int max_q, int max_kv,
                       int max_pages, int window, int sinks)
{
    constexpr int SMS = 152;
    AttendPlan p = {};
    const int group = heads / kv_heads;
    max_q = max_q < ntok ? max_q : ntok;
    // no sequence has more pages than its row of the table, whatever max_kv says: parts past
    // them would only fill the workspace
    long long pages = (static_cast<long long>(max_kv) + KV_PAGE - 1) / KV_PAGE;
    pages = pages < max_pages ? pages : max_pages;
    if (window > 0) {
        const long long seen = (static_cast<long long>(window) + max_q + sinks) / KV_PAGE + 3;
        pages = pages < seen ? pages : seen;
    }
    const long long rows = static_cast<long long>(max_q) * group;
    // The step kernel reads and widens the cache once per tile of 8 or 16 rows, the prompt kernel
    // once per 256, at a cost that hardly depends on how many there are.  Measured, us, step /
    // prompt kernel, 16 sequences of 8192 keys and 4 kv heads: f32 rows of 128 values, 32 rows
    // 86 / 95, 36 rows 113 / 96; 16-bit ones 16 rows 30 / 50, 24 rows 54 / 50; f32 rows of 64,
    // 24 rows 45 / 50, 32 rows 58 / 51; 16-bit ones 32 rows 34 / 45, 48 rows 45 / 45.
    const int few = dtype == KV_F32 ? (dim == 128 ? 32 : 24) : (dim == 128 ? 16 : 48);
    p.kernel = rows > few ? 1 : 0;
    // units: independent CTAs without parts; slots: CTAs that the chip holds at once; least, most:
    // pages of a part
    long long units, slots = SMS, parts, least, most;
    if (p.kernel == 0) {
        p.tile_rows = dtype == KV_F32 || rows <= 8 ? 8 : 16;
        p.row_tiles = static_cast<int>((rows + p.tile_rows - 1) / p.tile_rows);
        units = static_cast<long long>(batch) * kv_heads * p.row_tiles;
        slots = (p.tile_rows == 16 ? 3 : dim == 128 ? 4 : 6) * SMS;
        parts = slots / units;
        parts = parts < 1 ? 1 : parts;
        least = 4;      // a page a warp
        most = 64;      // sequences of uneven length: parts even the load out
    } else {
        // sum over the sequences of ceil(rows / KV_PROMPT_ROWS), or more
        const long long tiles =
            static_cast<long long>(ntok) * group / KV_PROMPT_ROWS + (batch < ntok ? batch : ntok);
        p.row_tiles = static_cast<int>(tiles < 0x7fffffffll ? tiles : 0x7fffffffll);
        units = tiles * kv_heads;
        // Where the tiles do not fill the chip, parts do, and cost the trip of their sums through
        // memory: the least of the expected times in us (GB300: a CTA's start and end 8; 128 keys
        // of 256 rows 3.0 for f32 rows of 128 values, 1.8 for 16-bit ones, half of it for 64
        // values; the join 8, most of it the host's, and its bytes at 6 TB/s).  More tiles than
        // SMs are left whole: two parts against the uneven last round took 821 us for 747 (2048
        // and 1944 tokens on 16384 and 13563, 32 heads on 8).
        const double step = (dtype == KV_F32 ? 3.0 : 1.8) * dim / 128;
        const double bytes = 8.0 * ntok * heads * dim;
        long long best = 1;
        double least_us = 0;
        for (long long n = 1; n == 1 || (units < SMS && n <= 64 && pages >= 8 * n); ++n) {
            const double us = static_cast<double>((units * n + SMS - 1) / SMS) * (8 + step * pages / 2 / n) +
                              (n == 1 ? 0 : 8 + n * bytes / 6e6);
            if (n == 1 || us < least_us) {
                best = n;
                least_us = us;
            }
        }
        parts = best;
        least = 8;
        // 16-bit rows: a sum in tensor memory, cut toward zero by every product, lost 3.9e-4 of
        // values of one sign after 65536 keys.  32768 keys stay below half a unit of f16's last
        // place, 131072 of bf16's; f32 rows move such sums out.
        most = dtype == KV_F16 ? 512 : dtype == KV_BF16 ? 2048 : 1ll << 30;
    }
    long long part = (pages + parts - 1) / parts;
    part = part < least ? least : part > most ? most : part;
    part = (part + 3) / 4 * 4;
    long long cut = (pages + part - 1) / part;
    p.cluster = 1;
    if (p.kernel == 0) {
        // Parts of half the chip or less become one cluster: no second kernel and no workspace (17
        // us for 22 for a call on 4 sequences of 1000 keys, most of it the host's), for up to 16
        // pieces at twice the pages.  A fuller chip has no room for clusters to fall into place
        // (64 clusters of 7 took 49 us where 448 CTAs took 30), and takes the join.
        const long long eighth = (pages + KV_MAX_CLUSTER - 1) / KV_MAX_CLUSTER;
        if (cut > KV_MAX_CLUSTER && cut <= 2 * KV_MAX_CLUSTER && units * KV_MAX_CLUSTER <= slots / 2) {
            part = (eighth + 3) / 4 * 4;
            cut = (pages + part - 1) / part;
        }
        if (cut <= KV_MAX_CLUSTER && units * cut <= slots / 2)
            p.cluster = static_cast<int>(cut);
    }
    p.part_pages = static_cast<int>(part * p.cluster);
    p.nsplit = static_cast<int>((pages + p.part_pages - 1) / p.part_pages);
    if (p.nsplit > 1) {
        const size_t flat = static_cast<size_t>(p.nsplit) * ntok * heads;
        p.part_bytes = flat * dim * sizeof(float);
        p.ml_bytes = (flat * sizeof(float2) + 15) / 16 * 16;
    }
    return p;
}

}  // namespace mmq

namespace {

using mmq::aligned;
using mmq::AttendPlan;
using mmq::KvRows;
using mmq::KvView;

mmq_status check_cache(const mmq_kv_cache* c)
{
    if (!c)
        return MMQ_ERR_ARG;
    if (c->head_dim != 64 && c->head_dim != 128)
        return MMQ_ERR_SHAPE;
    if (c->kv_heads < 1 || c->kv_heads > MMQ_KV_MAX_HEADS || c->num_pages < 1 || c->batch < 1 ||
        c->batch > MMQ_KV_MAX_BATCH || c->max_pages < 1 || c->max_pages > MMQ_KV_MAX_PAGES)
        return MMQ_ERR_SHAPE;
    if (!c->pages || !c->table || !c->start || !c->length)
        return MMQ_ERR_ARG;
    if (!aligned(c->pages, 16) || !aligned(c->table, 4) || !aligned(c->start, 4) || !aligned(c->length, 4))
        return MMQ_ERR_ALIGN;
    return MMQ_OK;
}

bool known_type(int t) { return t == MMQ_F32 || t == MMQ_F16 || t == MMQ_BF16; }

// [ntok][heads][dim] rows (no rows have no address); those that are written may not overlap.
mmq_status check_rows(const mmq_rows* r, int ntok, int heads, int dim, bool written)
{
    if (!r || (!r->data && ntok > 0) || !known_type(r->dtype) || r->token_stride < 0 || r->head_stride < 0)
        return MMQ_ERR_ARG;
    constexpr long long MOST = 1ll << 40;
    if (r->token_stride > MOST || r->head_stride > MOST)
        return MMQ_ERR_SHAPE;
    if (!aligned(r->data, r->dtype == MMQ_F32 ? 4 : 2))
        return MMQ_ERR_ALIGN;
    if (written) {
        const long long t = r->token_stride, h = r->head_stride;
        const bool by_token = (heads == 1 || h >= dim) && (ntok == 1 || t >= (heads - 1) * h + dim);
        const bool by_head = (ntok == 1 || t >= dim) && (heads == 1 || h >= (ntok - 1) * t + dim);
        if (!by_token && !by_head)
            return MMQ_ERR_ARG;
    }
    return MMQ_OK;
}

// Whether accesses of `bytes` from multiples of so many on are aligned in every row.
bool wide(const mmq_rows* r, int bytes)
{
    const int n = bytes / (r->dtype == MMQ_F32 ? 4 : 2);
    return aligned(r->data, static_cast<uintptr_t>(bytes)) && r->token_stride % n == 0 && r->head_stride % n == 0;
}

KvRows rows(const mmq_rows* r) { return {r->data, r->token_stride, r->head_stride}; }

mmq_status view(const mmq_kv_cache* c, KvView* v)
{
    unsigned int* err = nullptr;
    const cudaError_t e = mmq::device_error_word(&err);
    if (e != cudaSuccess)
        return MMQ_ERR_CUDA;
    *v = {static_cast<uint8_t*>(c->pages), c->table, c->start, c->length, c->num_pages, c->kv_heads, c->batch,
          c->max_pages, err + 1};
    return MMQ_OK;
}

mmq_status move_rows(bool write, const mmq_kv_cache* c, const mmq_rows* k, const mmq_rows* v, int ntok,
                     mmq_stream_t s)
{
    mmq_status st = check_cache(c);
    if (st != MMQ_OK)
        return st;
    if (ntok < 0 || ntok > MMQ_MAX_M)
        return MMQ_ERR_SHAPE;
    for (const mmq_rows* r : {k, v})
        if ((st = check_rows(r, ntok, c->kv_heads, c->head_dim, !write)) != MMQ_OK)
            return st;
    if (k->dtype != v->dtype)
        return MMQ_ERR_ARG;
    if (ntok == 0)
        return MMQ_OK;
    if ((st = mmq::check_device()) != MMQ_OK)
        return st;
    KvView cv;
    if ((st = view(c, &cv)) != MMQ_OK)
        return st;
    const auto launch = write ? mmq::launch_kv_write : mmq::launch_kv_read;
    return mmq::from_cuda(launch(cv, c->head_dim, k->dtype, rows(k), rows(v), wide(k, 16) && wide(v, 16), ntok,
                                 reinterpret_cast<cudaStream_t>(s)));
}

mmq_status check_attend(const mmq_kv_cache* c, int dtype, int heads, int ntok, int max_q, int max_kv, int window,
                        int sinks)
{
    if (!known_type(dtype) || window < 0 || sinks < 0 || max_q < 0 || max_kv < 0)
        return MMQ_ERR_ARG;
    if (c->head_dim != 64 && c->head_dim != 128)
        return MMQ_ERR_SHAPE;
    if (c->kv_heads < 1 || c->kv_heads > MMQ_KV_MAX_HEADS || c->batch < 1 || c->batch > MMQ_KV_MAX_BATCH ||
        c->max_pages < 1 || c->max_pages > MMQ_KV_MAX_PAGES || heads < 1 || heads > MMQ_KV_MAX_HEADS ||
        heads % c->kv_heads != 0 || ntok < 0 || ntok > MMQ_MAX_M)
        return MMQ_ERR_SHAPE;
    return MMQ_OK;
}

AttendPlan plan(const mmq_kv_cache* c, int dtype, int heads, int ntok, int max_q, int max_kv, int window, int sinks)
{
    return mmq::plan_attend(dtype, heads, c->kv_heads, c->head_dim, c->batch, ntok, max_q < 1 ? 1 : max_q,
                            max_kv < 1 ? 1 : max_kv, c->max_pages, window, sinks);
}

// What the weights need in the workspace beside the attention's: {reference, 1 / sum} of each row,
// then coefficients and scores of the step kernel, or many rows as operands.
struct WeighPlan {
    size_t stats_bytes, operand_bytes, score_bytes, coef_bytes;
    int cols, score_pages, score_rows;
    long long operand_rows;
};
WeighPlan weigh_plan(const mmq_kv_cache* c, const AttendPlan& attend, int dtype, int heads, int ntok, int max_q,
                     int max_kv)
{
    WeighPlan p = {};
    p.stats_bytes = (static_cast<size_t>(ntok) * static_cast<size_t>(heads) * sizeof(float2) + 15) / 16 * 16;
    p.operand_bytes = mmq::weigh_bytes(dtype, heads, c->kv_heads, c->head_dim, c->batch, ntok, max_q < 1 ? 1 : max_q,
                                       &p.cols, &p.operand_rows);
    // A few rows' scores are kept, unless they are more than a gigabyte (a batch of long tables without a
    // max_kv); the keys are then read again.  Kept / read again, us, attention included, 131071 keys of 8 kv
    // heads by rows a kv head: f32 rows of 128 values, 4 rows 56 / 78, 8 59 / 78, 16 99 / 114, 32 187 / 190; of 64, 4
    // 42 / 58, 8 47 / 59, 16 71 / 79, 24 103 / 104; f16 rows of 128, 4 52 / 73, 8 55 / 73, 16 67 / 77; of 64, 4 39 / 55, 8
    // 43 / 56, 16 54 / 56, 32 114 / 102, 48 150 / 123: from there on reading again would be the faster way.
    // 16 x 8191 keys give the same picture; 64 sequences of 95 to 8192, 4 bf16 rows of 128, 113 / 165.
    if (attend.kernel == 0) {
        const long long pages = (static_cast<long long>(max_kv < 1 ? 1 : max_kv) + mmq::KV_PAGE - 1) / mmq::KV_PAGE;
        p.score_pages = static_cast<int>(pages < c->max_pages ? pages : c->max_pages);
        p.score_rows = (max_q < 1 ? 1 : max_q < ntok ? max_q : ntok) * (heads / c->kv_heads);
        const size_t rows = static_cast<size_t>(c->batch) * c->kv_heads * p.score_rows;
        const size_t row = static_cast<size_t>(p.score_pages) * mmq::KV_PAGE * sizeof(float);
        if (rows <= (size_t{1} << 30) / row) {   // the product itself may pass 64 bits
            p.score_bytes = rows * row;
            p.coef_bytes = (rows * sizeof(float) + 15) / 16 * 16;
            p.operand_bytes = 0;
        }
    }
    return p;
}

struct Weights {
    const float* in;
    float* out;
    float decay;
};

mmq_status attend(const mmq_kv_cache* c, const mmq_rows* q, const mmq_rows* out, int heads, int ntok, int max_q,
                  int max_kv, float scale, int window, int sinks, const Weights* weights,
                  void* workspace, size_t workspace_bytes, mmq_stream_t s)
{
    mmq_status st = check_cache(c);
    if (st != MMQ_OK)
        return st;
    if (!q || !out)
        return MMQ_ERR_ARG;
    if ((st = check_attend(c, q->dtype, heads, ntok, max_q, max_kv, window, sinks)) != MMQ_OK ||
        (st = check_rows(q, ntok, heads, c->head_dim, false)) != MMQ_OK ||
        (st = check_rows(out, ntok, heads, c->head_dim, true)) != MMQ_OK)
        return st;
    // a positive normal number whose log2(e) multiple is finite
    if (q->dtype != out->dtype || !(scale >= 1.17549435e-38f && scale <= 1e38f))
        return MMQ_ERR_ARG;
    if (ntok == 0)
        return MMQ_OK;
    const AttendPlan p = plan(c, q->dtype, heads, ntok, max_q, max_kv, window, sinks);
    const WeighPlan wp = weights ? weigh_plan(c, p, q->dtype, heads, ntok, max_q, max_kv) : WeighPlan{};
    const size_t need = p.part_bytes + p.ml_bytes + wp.stats_bytes + wp.operand_bytes + wp.coef_bytes + wp.score_bytes;
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return MMQ_ERR_ARG;
        if (!aligned(workspace, 16))
            return MMQ_ERR_ALIGN;
    }
    // the grid: the units and a block (a cluster) for the rows of none
    if ((static_cast<long long>(p.nsplit) * p.row_tiles * c->kv_heads * (p.kernel == 0 ? c->batch : 1) + 1) * p.cluster >
            0x7fffffffll ||
        static_cast<long long>(ntok) * heads > 0x7fffffffll)
        return MMQ_ERR_SHAPE;
    if ((st = mmq::check_device()) != MMQ_OK)
        return st;
    mmq::AttendArgs a = {};
    if ((st = view(c, &a.c)) != MMQ_OK)
        return st;
    a.q = rows(q);
    a.out = rows(out);
    a.heads = heads;
    a.group = heads / c->kv_heads;
    a.ntok = ntok;
    a.scale_log2 = scale * 1.4426950408889634f;
    // positions are below 64 MMQ_KV_MAX_PAGES = 2^30, where larger windows and sinks change nothing
    constexpr int FAR = 1 << 30;
    a.window = window < FAR ? window : FAR;
    a.sinks = window == 0 ? 0 : sinks < FAR ? sinks : FAR;
    a.tile_rows = p.tile_rows;
    a.row_tiles = p.row_tiles;
    a.nsplit = p.nsplit;
    a.part_pages = p.part_pages;
    a.cluster = p.cluster;
    const int four = q->dtype == MMQ_F32 ? 16 : 8;   // bytes of four elements
    a.wide = wide(q, four) && wide(out, four);
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + p.part_bytes);
    uint8_t* rest = static_cast<uint8_t*>(workspace) + p.part_bytes + p.ml_bytes + wp.stats_bytes;
    if (weights)
        a.stats = reinterpret_cast<float2*>(rest - wp.stats_bytes);
    if (wp.score_bytes > 0) {
        a.coef = reinterpret_cast<float*>(rest);
        a.scores = reinterpret_cast<float*>(rest + wp.coef_bytes);
        a.score_pages = wp.score_pages;
        a.score_rows = wp.score_rows;
    }
    a.wc = {a.c.bad - 1, mmq::WAIT_LIMIT_NS, -1};
    bool injected = false;
    if (p.cluster == 1 && mmq::take_wait_ctl(&a.wc, &injected) != cudaSuccess)   // a cluster barrier has no time limit
        return MMQ_ERR_CUDA;
    const auto launch = p.kernel == 0 ? mmq::launch_kv_step : mmq::launch_kv_prompt;
    cudaError_t e = launch(a, c->head_dim, q->dtype, reinterpret_cast<cudaStream_t>(s));
    if (e == cudaSuccess && p.nsplit > 1)
        e = mmq::launch_kv_join(a, c->head_dim, q->dtype, reinterpret_cast<cudaStream_t>(s));
    if (e == cudaSuccess && weights) {
        a.wc = {a.c.bad - 1, mmq::WAIT_LIMIT_NS, -1};
        const mmq::WeighArgs w = {a, weights->in, weights->out, weights->decay, max_q < 1 ? 1 : max_q, p.tile_rows, wp.cols,
                                  wp.operand_rows, rest, 1};
        const auto weigh = a.scores ? mmq::launch_kv_finish_weights : mmq::launch_kv_weigh;
        e = weigh(w, c->head_dim, q->dtype, max_kv, reinterpret_cast<cudaStream_t>(s));
    }
    return mmq::from_cuda(e);
}

mmq_status check_plan(const mmq_rope_plan* p, int head_dim, mmq::RopeView* r)
{
    if (!p || !p->turns || (p->interleaved != 0 && p->interleaved != 1) || !std::isfinite(p->magnitude))
        return MMQ_ERR_ARG;
    if (p->rot_dim < 2 || p->rot_dim % 2 != 0 || p->rot_dim > head_dim)
        return MMQ_ERR_SHAPE;
    if (!aligned(p->turns, 8))
        return MMQ_ERR_ALIGN;
    *r = {reinterpret_cast<const unsigned long long*>(p->turns), p->rot_dim, p->interleaved != 0, p->magnitude};
    return MMQ_OK;
}

}  // namespace

extern "C" {

mmq_status mmq_kv_page_bytes(int kv_heads, int head_dim, size_t* bytes)
{
    if (!bytes)
        return MMQ_ERR_ARG;
    if (kv_heads < 1 || kv_heads > MMQ_KV_MAX_HEADS || (head_dim != 64 && head_dim != 128))
        return MMQ_ERR_SHAPE;
    *bytes = static_cast<size_t>(kv_heads) * head_dim * 72;
    return MMQ_OK;
}

mmq_status mmq_kv_write(const mmq_kv_cache* c, const mmq_rows* k, const mmq_rows* v, int ntok, mmq_stream_t s)
{
    return move_rows(true, c, k, v, ntok, s);
}

mmq_status mmq_kv_read(const mmq_kv_cache* c, const mmq_rows* k, const mmq_rows* v, int ntok, mmq_stream_t s)
{
    return move_rows(false, c, k, v, ntok, s);
}

mmq_status mmq_kv_attend_workspace_bytes(const mmq_kv_cache* c, int dtype, int heads, int ntok, int max_q, int max_kv,
                                         int window, int sinks, size_t* bytes)
{
    if (!c || !bytes)
        return MMQ_ERR_ARG;
    const mmq_status st = check_attend(c, dtype, heads, ntok, max_q, max_kv, window, sinks);
    if (st != MMQ_OK)
        return st;
    *bytes = 0;
    if (ntok > 0) {
        const AttendPlan p = plan(c, dtype, heads, ntok, max_q, max_kv, window, sinks);
        *bytes = p.part_bytes + p.ml_bytes;
    }
    return MMQ_OK;
}

mmq_status mmq_kv_attend(const mmq_kv_cache* c, const mmq_rows* q, const mmq_rows* out, int heads, int ntok, int max_q,
                         int max_kv, float scale, int window, int sinks, void* workspace, size_t workspace_bytes,
                         mmq_stream_t s)
{
    return attend(c, q, out, heads, ntok, max_q, max_kv, scale, window, sinks, nullptr, workspace, workspace_bytes, s);
}

mmq_status mmq_kv_attend_weights_workspace_bytes(const mmq_kv_cache* c, int dtype, int heads, int ntok, int max_q,
                                                 int max_kv, int window, int sinks, size_t* bytes)
{
    const mmq_status st = mmq_kv_attend_workspace_bytes(c, dtype, heads, ntok, max_q, max_kv, window, sinks, bytes);
    if (st == MMQ_OK && ntok > 0) {
        const WeighPlan p = weigh_plan(c, plan(c, dtype, heads, ntok, max_q, max_kv, window, sinks), dtype, heads, ntok, max_q,
                                       max_kv);
        *bytes += p.stats_bytes + p.operand_bytes + p.coef_bytes + p.score_bytes;
    }
    return st;
}

mmq_status mmq_kv_attend_weights(const mmq_kv_cache* c, const mmq_rows* q, const mmq_rows* out, int heads, int ntok,
                                 int max_q, int max_kv, float scale, int window, int sinks, const float* weights,
                                 float* new_weights, float decay, void* workspace, size_t workspace_bytes,
                                 mmq_stream_t s)
{
    if (!weights || !new_weights || !(decay >= 0.0f && decay <= 1.0f))
        return MMQ_ERR_ARG;
    if (!aligned(weights, 16) || !aligned(new_weights, 16))
        return MMQ_ERR_ALIGN;
    const Weights w = {weights, new_weights, decay};
    return attend(c, q, out, heads, ntok, max_q, max_kv, scale, window, sinks, &w, workspace, workspace_bytes, s);
}

mmq_status mmq_kv_evict(const mmq_kv_cache* c, float* weights, const int32_t* new_table, int new_pages, int keep,
                        int first, int last, int max_kv, int32_t* new_length, int32_t* kept, mmq_stream_t s)
{
    mmq_status st = check_cache(c);
    if (st != MMQ_OK)
        return st;
    if (!weights || !new_table || !new_length || !kept || first < 0 || last < 0 || max_kv < 0)
        return MMQ_ERR_ARG;
    if (keep < 1 || new_pages < 1 || new_pages > MMQ_KV_MAX_PAGES ||
        static_cast<long long>(new_pages) * mmq::KV_PAGE < keep || static_cast<long long>(first) + last > keep)
        return MMQ_ERR_SHAPE;
    if (!aligned(weights, 16) || !aligned(new_table, 4) || !aligned(new_length, 4) || !aligned(kept, 4))
        return MMQ_ERR_ALIGN;
    // grids: CTAs of the choice, new pages of the move
    const long long units = static_cast<long long>(c->batch) * c->kv_heads;
    if (units * ((keep + mmq::KV_PAGE - 1) / mmq::KV_PAGE) > 0x7fffffffll)
        return MMQ_ERR_SHAPE;
    if ((st = mmq::check_device()) != MMQ_OK)
        return st;
    mmq::EvictArgs a = {};
    if ((st = view(c, &a.c)) != MMQ_OK)
        return st;
    a.weights = weights;
    a.new_table = new_table;
    a.new_length = new_length;
    a.kept = kept;
    a.new_pages = new_pages;
    a.keep = keep;
    a.first = first;
    a.last = last;
    return mmq::from_cuda(mmq::launch_kv_evict(a, c->head_dim, max_kv, reinterpret_cast<cudaStream_t>(s)));
}

mmq_status mmq_rope_frequencies(mmq_rope_scaling scaling, int rot_dim, double base, double factor, double original,
                                double* freq, float* magnitude)
{
    if (!freq || !magnitude || !(base > 1.0 && std::isfinite(base)))
        return MMQ_ERR_ARG;
    if (rot_dim < 2 || rot_dim > MMQ_ROPE_MAX_DIM || rot_dim % 2 != 0)
        return MMQ_ERR_SHAPE;
    if (scaling < MMQ_ROPE_PLAIN || scaling > MMQ_ROPE_BANDS)
        return MMQ_ERR_ARG;
    if (scaling != MMQ_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor)))
        return MMQ_ERR_ARG;
    if (scaling >= MMQ_ROPE_YARN && !(original >= 1.0 && std::isfinite(original)))
        return MMQ_ERR_ARG;
    constexpr double PI = 3.14159265358979323846;
    const int half = rot_dim / 2;
    *magnitude = 1.0f;
    if (scaling == MMQ_ROPE_NTK && rot_dim > 2) {
        base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
        if (!std::isfinite(base))
            return MMQ_ERR_ARG;
    }
    // YaRN's ramp between the pairs that make 32 turns and 1 turn in the original context
    double lo = 0.0, hi = 0.0;
    if (scaling == MMQ_ROPE_YARN) {
        const auto pair = [&](double turns) {
            return rot_dim * std::log(original / (turns * 2.0 * PI)) / (2.0 * std::log(base));
        };
        const auto limit = [&](double d) { return d < 0.0 ? 0.0 : d > rot_dim - 1.0 ? rot_dim - 1.0 : d; };
        lo = limit(std::floor(pair(32.0)));
        hi = limit(std::ceil(pair(1.0)));
        *magnitude = static_cast<float>(0.1 * std::log(factor) + 1.0);
    }
    for (int i = 0; i < half; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == MMQ_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == MMQ_ROPE_YARN) {
            const double width = hi - lo > 0.001 ? hi - lo : 0.001;
            double ramp = (i - lo) / width;
            ramp = ramp < 0.0 ? 0.0 : ramp > 1.0 ? 1.0 : ramp;
            f = f / factor * ramp + f * (1.0 - ramp);
        } else if (scaling == MMQ_ROPE_BANDS) {
            double near = (original * f / (2.0 * PI) - 1.0) / 3.0;
            near = near < 0.0 ? 0.0 : near > 1.0 ? 1.0 : near;
            f = (1.0 - near) * f / factor + near * f;
        }
        freq[i] = f;
    }
    return MMQ_OK;
}

mmq_status mmq_rope_turns(const double* freq, int n, uint64_t* turns)
{
    if (!freq || !turns)
        return MMQ_ERR_ARG;
    if (n < 1 || n > MMQ_ROPE_MAX_DIM / 2)
        return MMQ_ERR_SHAPE;
    for (int i = 0; i < n; ++i)
        if (!(std::fabs(freq[i]) <= 1e6))
            return MMQ_ERR_ARG;
    // 1 / (2 pi) in two parts; a product's two parts are below 2^18, its error below 2^-88
    constexpr double HI = 0.15915494309189535, LO = -9.839338337591243e-18;
    for (int i = 0; i < n; ++i) {
        const double f = std::fabs(freq[i]), p = f * HI, q = std::fma(f, HI, -p) + f * LO;
        const double whole = std::ldexp(p - std::floor(p), 64);   // below 2^64; cut to a whole number
        const double rest = whole - std::floor(whole) + std::ldexp(q, 64);
        const uint64_t w = static_cast<uint64_t>(whole) + static_cast<uint64_t>(static_cast<int64_t>(std::nearbyint(rest)));
        turns[i] = freq[i] < 0.0 ? ~w + 1u : w;
    }
    return MMQ_OK;
}

mmq_status mmq_rope(const mmq_rope_plan* p, const mmq_rows* x, const mmq_rows* out, const int32_t* pos, int heads,
                    int head_dim, int ntok, mmq_stream_t s)
{
    mmq::RopeView r;
    mmq_status st = check_plan(p, head_dim, &r);
    if (st != MMQ_OK)
        return st;
    if (!pos && ntok > 0)
        return MMQ_ERR_ARG;
    if (heads < 1 || heads > MMQ_KV_MAX_HEADS || head_dim > MMQ_ROPE_MAX_DIM || ntok < 0 || ntok > MMQ_MAX_M)
        return MMQ_ERR_SHAPE;
    if ((st = check_rows(x, ntok, heads, head_dim, false)) != MMQ_OK ||
        (st = check_rows(out, ntok, heads, head_dim, true)) != MMQ_OK)
        return st;
    if (x->dtype != out->dtype)
        return MMQ_ERR_ARG;
    if (!aligned(pos, 4))
        return MMQ_ERR_ALIGN;
    if (ntok == 0)
        return MMQ_OK;
    if ((st = mmq::check_device()) != MMQ_OK)
        return st;
    return mmq::from_cuda(mmq::launch_rope(rows(x), rows(out), pos, r, x->dtype, heads, head_dim, ntok,
                                           wide(x, 16) && wide(out, 16), reinterpret_cast<cudaStream_t>(s)));
}

mmq_status mmq_kv_write_rope(const mmq_kv_cache* c, const mmq_rope_plan* p, const mmq_rows* q, const mmq_rows* q_out,
                             int heads, const mmq_rows* k, const mmq_rows* v, const int32_t* pos, int ntok,
                             mmq_stream_t s)
{
    mmq_status st = check_cache(c);
    if (st != MMQ_OK)
        return st;
    mmq::RopeView r;
    if ((st = check_plan(p, c->head_dim, &r)) != MMQ_OK)
        return st;
    if (!pos && ntok > 0)
        return MMQ_ERR_ARG;
    if (heads < 1 || heads > MMQ_KV_MAX_HEADS || ntok < 0 || ntok > MMQ_MAX_M)
        return MMQ_ERR_SHAPE;
    if ((st = check_rows(q, ntok, heads, c->head_dim, false)) != MMQ_OK ||
        (st = check_rows(q_out, ntok, heads, c->head_dim, true)) != MMQ_OK)
        return st;
    for (const mmq_rows* x : {k, v})
        if ((st = check_rows(x, ntok, c->kv_heads, c->head_dim, false)) != MMQ_OK)
            return st;
    if (q->dtype != q_out->dtype || q->dtype != k->dtype || k->dtype != v->dtype)
        return MMQ_ERR_ARG;
    if (!aligned(pos, 4))
        return MMQ_ERR_ALIGN;
    if (ntok == 0)
        return MMQ_OK;
    if ((st = mmq::check_device()) != MMQ_OK)
        return st;
    mmq::KvView cv;
    if ((st = view(c, &cv)) != MMQ_OK)
        return st;
    return mmq::from_cuda(mmq::launch_kv_write_rope(cv, c->head_dim, q->dtype, rows(q), rows(q_out), heads, rows(k),
                                                    rows(v), pos, r, wide(q, 16) && wide(q_out, 16),
                                                    wide(k, 16) && wide(v, 16), ntok,
                                                    reinterpret_cast<cudaStream_t>(s)));
}

}  // extern "C"
