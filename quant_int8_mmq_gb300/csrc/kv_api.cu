// kv_api.cu -- entry points of the 4-bit key/value cache and the attention over it.
//
// As in api.cu, arguments are checked on the host before any CUDA call; what only the
// device knows (page ids, lengths) is checked by the kernels.
#include "api.h"
#include "kv.cuh"

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
    if (p.part_bytes + p.ml_bytes > 0) {
        if (!workspace || workspace_bytes < p.part_bytes + p.ml_bytes)
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
    a.wc = {a.c.bad - 1, mmq::WAIT_LIMIT_NS, -1};
    bool injected = false;
    if (p.cluster == 1 && mmq::take_wait_ctl(&a.wc, &injected) != cudaSuccess)   // a cluster barrier has no time limit
        return MMQ_ERR_CUDA;
    const auto launch = p.kernel == 0 ? mmq::launch_kv_step : mmq::launch_kv_prompt;
    cudaError_t e = launch(a, c->head_dim, q->dtype, reinterpret_cast<cudaStream_t>(s));
    if (e == cudaSuccess && p.nsplit > 1)
        e = mmq::launch_kv_join(a, c->head_dim, q->dtype, reinterpret_cast<cudaStream_t>(s));
    return mmq::from_cuda(e);
}

}  // extern "C"
