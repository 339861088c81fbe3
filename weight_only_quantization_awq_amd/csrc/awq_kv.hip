// C ABI of the 4-bit key/value cache: host-side validation, workspace layout
// and the choice of launches.  See include/awq.h for the contract.
#include "awq.h"  // include/awq.h (on the -I path)

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "kv_host.h"

namespace awq {

awq_status kv_fail(awq_status code, const char *fmt, ...) {
    char msg[384];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return static_cast<awq_status>(report_error(code, msg));
}

awq_status kv_hip_status(hipError_t e, const char *what) {
    if (e == hipSuccess) return AWQ_OK;
    return kv_fail(AWQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// A launch has fewer than 2^32 threads: dim/2 to a unit of the copy kernels, and on the
// wide path of the attention at most 512 to an item and to 256 of its columns.
static constexpr int64_t kMaxUnits = int64_t(1) << 25;   // (at dim 128)
static constexpr int64_t kMaxItems = int64_t(1) << 21;   // batch * heads

// The sizes of a cache: 0 or the bytes of one (page, head).
static int64_t block_bytes(int page, int64_t heads, int dim, int group) {
    if (dim != 64 && dim != 128 && dim != 256) {
        kv_fail(AWQ_ERR_SHAPE, "dim must be 64, 128 or 256 (got %d)", dim);
        return 0;
    }
    if ((group != 32 && group != 64 && group != 128) || group > dim) {
        kv_fail(AWQ_ERR_ARG, "group must be 32, 64 or 128 and at most dim (got %d)", group);
        return 0;
    }
    if (page < 16 || page > 256 || (page & (page - 1)) != 0) {
        kv_fail(AWQ_ERR_ARG, "page must be a power of two in 16..256 (got %d)", page);
        return 0;
    }
    if (heads < 1 || heads > 65535) {
        kv_fail(AWQ_ERR_SHAPE, "heads must be in 1..65535 (got %lld)", static_cast<long long>(heads));
        return 0;
    }
    return static_cast<int64_t>(page) * dim + 8ll * page * (dim / group);
}

size_t kv_page_bytes(int page, int64_t heads, int dim, int group) {
    return static_cast<size_t>(block_bytes(page, heads, dim, group) * heads);
}

awq_status kv_check(const awq_kv_cache *cache, const awq_kv_batch *batch, KvCache *c, KvBatch *s, bool sizes_only) {
    if (!cache || !batch) return kv_fail(AWQ_ERR_ARG, "cache and batch must be non-NULL");
    const int64_t block = block_bytes(cache->page, cache->heads, cache->dim, cache->group);
    if (block == 0) return cache->dim != 64 && cache->dim != 128 && cache->dim != 256 ? AWQ_ERR_SHAPE
                           : cache->heads < 1 || cache->heads > 65535                ? AWQ_ERR_SHAPE
                                                                                      : AWQ_ERR_ARG;
    if (batch->batch < 1 || batch->batch > kKvMaxCount) return kv_fail(AWQ_ERR_SHAPE, "batch must be >= 1");
    if (batch->rows < 0 || batch->rows > kKvMaxCount) return kv_fail(AWQ_ERR_SHAPE, "rows must be >= 0");
    if (batch->max_pages < 1 || batch->max_pages > kKvMaxCount || batch->max_pages * cache->page > kKvMaxCount)
        return kv_fail(AWQ_ERR_SHAPE, "max_pages must be >= 1 and hold at most 2^30 positions");
    if (!batch->row_start && batch->rows % batch->batch != 0)
        return kv_fail(AWQ_ERR_SHAPE, "without row_start, rows (%lld) must be a multiple of batch (%lld)",
                    static_cast<long long>(batch->rows), static_cast<long long>(batch->batch));
    const int64_t tiles = (batch->max_pages * cache->page + kKvTile - 1) / kKvTile;
    // units of the copy kernels, and tiles of the attention's line
    if ((batch->rows / 4 + 2 * batch->batch) * cache->heads > kMaxUnits * 128 / cache->dim ||
        batch->batch * cache->heads > kMaxItems ||
        batch->batch * cache->heads * (tiles + kKvItemCost) > kKvMaxCount)
        return kv_fail(AWQ_ERR_SHAPE, "batch * heads * max_pages or rows * heads too large for one call");
    int shift = 0;
    while ((1 << shift) < cache->page) ++shift;
    c->pages = static_cast<unsigned char *>(cache->pages);
    c->page_stride = cache->page_stride;
    c->block = block;
    c->n_pages = static_cast<int>(cache->n_pages);
    c->page_shift = shift;
    c->heads = static_cast<int>(cache->heads);
    c->dim = cache->dim;
    c->group = cache->group;
    s->row_start = batch->row_start;
    s->kv_len = batch->kv_len;
    s->table = batch->block_table;
    s->B = static_cast<int>(batch->batch);
    s->max_pages = static_cast<int>(batch->max_pages);
    s->T = static_cast<int>(batch->rows);
    s->even = static_cast<int>(batch->rows / batch->batch);
    if (sizes_only) return AWQ_OK;
    if (cache->n_pages < 1 || cache->n_pages > INT32_MAX) return kv_fail(AWQ_ERR_SHAPE, "n_pages must be in 1..2^31-1");
    if (cache->page_stride < cache->heads * block || cache->page_stride % 16 != 0)
        return kv_fail(AWQ_ERR_SHAPE, "page_stride must be a multiple of 16 and at least %lld bytes (got %lld)",
                    static_cast<long long>(cache->heads * block), static_cast<long long>(cache->page_stride));
    if (!cache->pages || !kv_aligned(cache->pages, 16)) return kv_fail(AWQ_ERR_ARG, "pages must be non-NULL, 16-byte aligned");
    if (!batch->kv_len || !batch->block_table) return kv_fail(AWQ_ERR_ARG, "kv_len and block_table must be non-NULL");
    if (!kv_aligned(batch->kv_len, 4) || !kv_aligned(batch->block_table, 4) || !kv_aligned(batch->row_start, 4))
        return kv_fail(AWQ_ERR_ARG, "row_start, kv_len and block_table must be 4-byte aligned");
    return AWQ_OK;
}

bool kv_wide_type(awq_dtype t) { return t == AWQ_F32 || t == AWQ_BF16 || t == AWQ_F16; }

awq_status kv_check_rows(const void *p, const char *name, awq_dtype t, int64_t rows, int64_t stride, int64_t least) {
    if (rows > 0 && !p) return kv_fail(AWQ_ERR_ARG, "%s must be non-NULL", name);
    if (!kv_aligned(p, 16)) return kv_fail(AWQ_ERR_ARG, "%s must be 16-byte aligned", name);
    const int64_t size = t == AWQ_F32 ? 4 : 2;
    if (stride < least || stride > kKvMaxCount || stride * size % 16 != 0)
        return kv_fail(AWQ_ERR_SHAPE, "the row stride of %s must be at least %lld elements and a multiple of 16 bytes "
                    "(got %lld)", name, static_cast<long long>(least), static_cast<long long>(stride));
    return AWQ_OK;
}

awq_status kv_check_copy(const awq_kv_cache *cache, const awq_kv_batch *batch, const void *K, const void *V, awq_dtype t,
                         int64_t k_stride, int64_t v_stride, KvCache *c, KvBatch *s) {
    report_error(AWQ_OK, "");
    awq_status e = kv_check(cache, batch, c, s);
    if (e != AWQ_OK) return e;
    if (!kv_wide_type(t)) return kv_fail(AWQ_ERR_DTYPE, "unsupported dtype %d", static_cast<int>(t));
    const int64_t least = cache->heads * cache->dim;
    if ((e = kv_check_rows(K, "K", t, batch->rows, k_stride, least)) != AWQ_OK) return e;
    return kv_check_rows(V, "V", t, batch->rows, v_stride, least);
}

}  // namespace awq

namespace {

using awq::kv_aligned;
using awq::kv_check;
using awq::kv_check_copy;
using awq::kv_check_rows;
using awq::kv_fail;
using awq::kv_hip_status;
using awq::kKvMaxCount;

// The launches of one attention call and its workspace (byte offsets).
struct Plan {
    bool split, wide, merge, line, wide_merge, apart;
    int snap, tiles_col, split_cols, workers, units, own_units, line_units, wide_workers;
    size_t items, part_ml, part, wide_items, wide_ml, wide_part, own_ml, own, common_ml, common, total;
};

constexpr int kSimds = 4 * awq::kKvCus;

// prefix: the sequence of all rows over a shared prefix, or NULL.
awq_status plan(const awq::KvCache &c, const awq::KvBatch &s, int64_t q_heads, int64_t max_rows, const awq::KvBatch *prefix, Plan *p) {
    if (q_heads < 1 || q_heads > 65535 || q_heads % c.heads != 0)
        return kv_fail(AWQ_ERR_SHAPE, "q_heads (%lld) must be a multiple of the cache's heads (%d)",
                    static_cast<long long>(q_heads), c.heads);
    if (max_rows < 0) return kv_fail(AWQ_ERR_SHAPE, "max_rows must be >= 0");
    if (static_cast<int64_t>(s.T) * q_heads > kKvMaxCount) return kv_fail(AWQ_ERR_SHAPE, "rows * q_heads too large for one call");
    // (the join of a call with a prefix: dim/4 threads to a row and query head)
    if (prefix && static_cast<int64_t>(s.T) * q_heads * c.dim / 4 >= int64_t(1) << 32)
        return kv_fail(AWQ_ERR_SHAPE, "rows * q_heads too large for one call with a prefix");
    const int64_t per = q_heads / c.heads;
    const int64_t most = s.row_start ? (max_rows == 0 || max_rows > s.T ? s.T : max_rows) : s.even;
    const int64_t cols = most * per, all_cols = prefix ? s.T * per : 0, limit = awq::kv_split_cols(c.dim);
    const int64_t positions = static_cast<int64_t>(s.max_pages) << c.page_shift;
    const int64_t all_positions = prefix ? static_cast<int64_t>(prefix->max_pages) << c.page_shift : 0;
    auto in = [](int64_t n, int64_t size) { return (n + size - 1) / size; };
    *p = Plan{};
    const bool own_wide = cols > limit, all_wide = all_cols > limit, all_split = prefix && !all_wide;
    p->wide = own_wide || all_wide;
    // Where the sequences take the wide path, the split path is for their single tokens.
    // With a prefix whose columns take it, one launch serves its items and the sequences', with the
    // column tiles that the prefix needs.  (That costs where own parts are long: single tokens, 32 query
    // heads on 8 of dim 128, 4096 positions of their own behind 512, us of a call: 8 sequences, two tiles, 27;
    // 9, four tiles, 43; 16 66; 17, whose prefix takes the wide path and whose own items one tile, 57; over one
    // table 21, 21, 29 and 29.)
    const int64_t need = own_wide ? per : all_split ? all_cols : cols;
    p->split = need <= limit && (!own_wide || s.row_start);
    p->tiles_col = need <= 16 ? 1 : need <= 32 ? 2 : 4;
    // What a sequence's columns are compared with on the device is what the workspace holds for
    // each piece: one with more rows than max_rows is left out, not kept in too small a place.
    p->split_cols = p->split ? static_cast<int>(own_wide ? 16 * p->tiles_col : need) : 0;
    const int64_t own_tiles = in(positions, awq::kKvTile), all_tiles = all_split ? in(all_positions, awq::kKvTile) : 0;
    const int64_t tiles = own_tiles > all_tiles ? own_tiles : all_tiles;
    const int64_t line = c.heads * (s.B * (own_tiles + awq::kKvItemCost) + (all_split ? all_tiles + awq::kKvItemCost : 0));
    if (line > kKvMaxCount) return kv_fail(AWQ_ERR_SHAPE, "batch * heads * pages too large for one call");
    const int64_t useful = in(line, awq::kKvMinShare);
    const int64_t fill = kSimds * awq::kv_split_waves(c.dim, p->tiles_col);
    p->workers = static_cast<int>(useful < fill ? useful : fill);
    p->snap = static_cast<int>(tiles <= awq::kKvWhole ? tiles : awq::kKvSnap);
    p->merge = p->split && tiles > 2 * p->snap + 1;   // shorter items are never cut
    const int64_t wide = awq::kv_wide_cols(c.dim), tile = awq::kv_wide_tile(c.dim);
    p->own_units = !own_wide ? 0 : static_cast<int>(s.row_start ? s.T * per / wide + s.B : s.B * in(s.even * per, wide));
    const int64_t all_units = all_wide ? in(all_cols, wide) : 0;
    p->units = static_cast<int>(p->own_units + all_units);
    const int64_t own_wide_tiles = own_wide ? in(positions, tile) : 0, all_wide_tiles = all_wide ? in(all_positions, tile) : 0;
    // Where the sequences' units are too many for a line and the prefix's are not, the prefix's form
    // one by themselves, in a launch of their own.
    p->apart = p->own_units * c.heads >= awq::kKvLineUnits && all_units > 0 && all_units * c.heads < awq::kKvLineUnits;
    const int64_t own_on_line = p->apart ? 0 : p->own_units;
    p->line_units = static_cast<int>(own_on_line + all_units);
    const int64_t groups = static_cast<int64_t>(p->line_units) * c.heads;
    const int64_t wide_tiles = own_wide_tiles > all_wide_tiles && !p->apart ? own_wide_tiles : all_wide_tiles;
    const int64_t wide_line = c.heads * (own_on_line * (own_wide_tiles + awq::kv_wide_cost(c.dim)) +
                                         all_units * (all_wide_tiles + awq::kv_wide_cost(c.dim)));
    p->line = p->wide && groups < awq::kKvLineUnits && wide_line <= kKvMaxCount;
    const int64_t wide_useful = in(wide_line, awq::kKvWideMinShare);
    p->wide_workers = static_cast<int>(wide_useful < awq::kKvCus ? wide_useful : awq::kKvCus);
    p->wide_merge = p->line && wide_tiles > 2 * awq::kKvWideSnap + 1;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    if (p->merge) {
        const size_t n = static_cast<size_t>(p->workers) * 2 * p->split_cols;
        p->items = take((static_cast<size_t>(s.B) + (prefix ? 1 : 0)) * c.heads * 8);
        p->part_ml = take(n * 8);
        p->part = take(n * c.dim * 4);
    }
    if (p->wide_merge) {
        const size_t n = static_cast<size_t>(p->wide_workers) * 2 * wide;
        p->wide_items = take(static_cast<size_t>(groups) * 8);
        p->wide_ml = take(n * 8);
        p->wide_part = take(n * c.dim * 4);
    }
    if (prefix) {
        const size_t heads = static_cast<size_t>(s.T) * static_cast<size_t>(q_heads);
        p->own_ml = take(heads * 8);
        p->own = take(heads * c.dim * 4);
        p->common_ml = take(heads * 8);
        p->common = take(heads * c.dim * 4);
    }
    p->total = at;
    return AWQ_OK;
}

// The prefix of a view as the kernels take it, in *all; false: refused.
awq_status check_prefix(const awq_kv_cache *cache, const awq_kv_batch *batch, const awq_kv_view *view, awq::KvBatch *all) {
    awq_kv_batch one = *batch;
    one.batch = 1;
    one.max_pages = view->prefix_pages;
    one.row_start = nullptr;
    one.kv_len = view->prefix_len;
    one.block_table = view->prefix_table;
    if (view->prefix_pages < 1 || view->prefix_pages > kKvMaxCount)
        return kv_fail(AWQ_ERR_SHAPE, "prefix_pages must be >= 1 (got %lld)", static_cast<long long>(view->prefix_pages));
    awq::KvCache c;
    return kv_check(cache, &one, &c, all, true);
}

awq_status plan_call(const awq::KvAttend &a, const awq_kv_cache *cache, const awq_kv_batch *batch, const awq_kv_view *view,
                     int64_t q_heads, int64_t max_rows, awq::KvBatch *all, Plan *p) {
    if (!view) return kv_fail(AWQ_ERR_ARG, "view must be non-NULL");
    if (!view->prefix_len) return plan(a.c, a.s, q_heads, max_rows, nullptr, p);
    const awq_status e = check_prefix(cache, batch, view, all);
    return e != AWQ_OK ? e : plan(a.c, a.s, q_heads, max_rows, all, p);
}

}  // namespace

extern "C" {

size_t awq_kv_page_size(int page, int64_t heads, int dim, int group) {
    awq::report_error(AWQ_OK, "");
    return awq::kv_page_bytes(page, heads, dim, group);
}

awq_status awq_kv_append(const awq_kv_cache *cache, const awq_kv_batch *batch, const void *K, const void *V,
                         awq_dtype t, int64_t k_stride, int64_t v_stride, hipStream_t stream) {
    awq::KvCache c{};
    awq::KvBatch s{};
    const awq_status e = kv_check_copy(cache, batch, K, V, t, k_stride, v_stride, &c, &s);
    if (e != AWQ_OK || s.T == 0) return e;
    return kv_hip_status(awq::launch_kv_append(c, s, K, V, t, k_stride, v_stride, stream), "awq_kv_append launch");
}

awq_status awq_kv_read(const awq_kv_cache *cache, const awq_kv_batch *batch, void *K, void *V, awq_dtype t,
                       int64_t k_stride, int64_t v_stride, hipStream_t stream) {
    awq::KvCache c{};
    awq::KvBatch s{};
    const awq_status e = kv_check_copy(cache, batch, K, V, t, k_stride, v_stride, &c, &s);
    if (e != AWQ_OK || s.T == 0) return e;
    return kv_hip_status(awq::launch_kv_read(c, s, K, V, t, k_stride, v_stride, stream), "awq_kv_read launch");
}

size_t awq_kv_attention_workspace_size_ex(const awq_kv_cache *cache, const awq_kv_batch *batch, const awq_kv_view *view,
                                          int64_t q_heads, int64_t max_rows) {
    awq::report_error(AWQ_OK, "");
    awq::KvAttend a{};
    awq::KvBatch all{};
    Plan p{};
    if (kv_check(cache, batch, &a.c, &a.s, true) != AWQ_OK ||
        plan_call(a, cache, batch, view, q_heads, max_rows, &all, &p) != AWQ_OK)
        return 0;
    return p.total;
}

size_t awq_kv_attention_workspace_size(const awq_kv_cache *cache, const awq_kv_batch *batch, int64_t q_heads,
                                       int64_t max_rows) {
    const awq_kv_view view{};
    return awq_kv_attention_workspace_size_ex(cache, batch, &view, q_heads, max_rows);
}

awq_status awq_kv_attention_ex(const awq_kv_cache *cache, const awq_kv_batch *batch, const awq_kv_view *view, const void *Q,
                               awq_dtype t, int64_t q_heads, int64_t q_stride, int64_t max_rows, float scale, int causal, void *O,
                               int64_t o_stride, float *lse, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    awq::report_error(AWQ_OK, "");
    awq::KvAttend a{};
    awq::KvBatch all{};
    Plan p{};
    awq_status e = kv_check(cache, batch, &a.c, &a.s);
    if (e != AWQ_OK) return e;
    if (t != AWQ_BF16 && t != AWQ_F16) return kv_fail(AWQ_ERR_DTYPE, "Q must be AWQ_BF16 or AWQ_F16 (got %d)", static_cast<int>(t));
    if ((e = plan_call(a, cache, batch, view, q_heads, max_rows, &all, &p)) != AWQ_OK) return e;
    const int64_t least = q_heads * cache->dim;
    if ((e = kv_check_rows(Q, "Q", t, batch->rows, q_stride, least)) != AWQ_OK) return e;
    if ((e = kv_check_rows(O, "O", t, batch->rows, o_stride, least)) != AWQ_OK) return e;
    if (!kv_aligned(lse, 4)) return kv_fail(AWQ_ERR_ARG, "lse must be 4-byte aligned");
    if (!(scale > 0.0f) || !isfinite(scale)) return kv_fail(AWQ_ERR_ARG, "scale must be positive and finite (got %g)", scale);
    if (causal != 0 && causal != 1) return kv_fail(AWQ_ERR_ARG, "causal must be 0 or 1 (got %d)", causal);
    const int64_t window = view->window, sinks = view->sinks;
    if (window < 0) return kv_fail(AWQ_ERR_ARG, "window must be >= 0 (0: none)");
    if (window > 0 && !causal) return kv_fail(AWQ_ERR_ARG, "a window needs causal = 1");
    if (sinks < 0) return kv_fail(AWQ_ERR_ARG, "sinks must be >= 0 (0: none)");
    if (sinks > 0 && window == 0) return kv_fail(AWQ_ERR_ARG, "sinks need a window");
    if (view->prefix_len) {
        if (window > 0) return kv_fail(AWQ_ERR_ARG, "a shared prefix and a window exclude each other");
        if (!view->prefix_table || !kv_aligned(view->prefix_table, 4) || !kv_aligned(view->prefix_len, 4))
            return kv_fail(AWQ_ERR_ARG, "prefix_table and prefix_len must be non-NULL, 4-byte aligned");
    }
    if (batch->rows == 0) return AWQ_OK;
    if (p.total > 0) {
        if (!workspace) return kv_fail(AWQ_ERR_WORKSPACE, "workspace is NULL (need %zu bytes)", p.total);
        if (!kv_aligned(workspace, 16)) return kv_fail(AWQ_ERR_WORKSPACE, "workspace must be 16-byte aligned");
        if (workspace_bytes < p.total)
            return kv_fail(AWQ_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", workspace_bytes, p.total);
    }
    // (in place, each query is read by those who write there, or by a launch before)
    if ((O != Q || (o_stride != q_stride && batch->rows > 1)) &&
        awq::kv_rows_meet({O, o_stride * 2, least * 2}, {Q, q_stride * 2, least * 2}, batch->rows))
        return kv_fail(AWQ_ERR_ARG, "O may be Q, of one row stride, but else must not share memory with it");
    a.Q = Q;
    a.O = O;
    a.lse = lse;
    a.q_stride = q_stride;
    a.o_stride = o_stride;
    a.q_heads = static_cast<int>(q_heads);
    a.per = a.q_heads / a.c.heads;
    a.scale_log2 = scale * 1.44269504088896341f;
    a.causal = causal;
    a.window = window > (int64_t(1) << 30) ? 0 : static_cast<int>(window);   // (no sequence is longer)
    a.split_cols = p.split_cols;
    a.tiles_col = p.tiles_col;
    a.workers = p.workers;
    a.snap = p.snap;
    a.units = p.units;
    a.line = p.line;
    a.wide_workers = p.wide_workers;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    auto floats = [&](size_t at) { return reinterpret_cast<float *>(ws + at); };
    if (p.merge) {
        a.items = reinterpret_cast<int2 *>(ws + p.items);
        a.part_ml = floats(p.part_ml);
        a.part = floats(p.part);
    }
    if (p.wide_merge) {
        a.wide_items = reinterpret_cast<int2 *>(ws + p.wide_items);
        a.wide_ml = floats(p.wide_ml);
        a.wide_part = floats(p.wide_part);
    }
    awq::KvView v{};
    v.sinks = a.window == 0 ? 0 : static_cast<int>(sinks > kKvMaxCount ? kKvMaxCount : sinks);
    if (view->prefix_len)
        v.prefix = {view->prefix_len, view->prefix_table, all.max_pages, p.own_units, p.apart ? p.own_units : 0, floats(p.own), floats(p.own_ml),
                    floats(p.common), floats(p.common_ml)};
    if (v.sinks > 0 || view->prefix_len) a.view = &v;
    hipError_t h;
    if (a.c.dim == 64)
        h = awq::launch_kv_attend_64(a, t, p.split, p.wide, p.merge, stream);
    else if (a.c.dim == 128)
        h = awq::launch_kv_attend_128(a, t, p.split, p.wide, p.merge, stream);
    else
        h = awq::launch_kv_attend_256(a, t, p.split, p.wide, p.merge, stream);
    return kv_hip_status(h, "awq_kv_attention launch");
}

awq_status awq_kv_attention(const awq_kv_cache *cache, const awq_kv_batch *batch, const void *Q, awq_dtype t,
                            int64_t q_heads, int64_t q_stride, int64_t max_rows, float scale, int causal,
                            int64_t window, void *O, int64_t o_stride, float *lse, void *workspace,
                            size_t workspace_bytes, hipStream_t stream) {
    awq_kv_view view{};
    view.window = window;
    return awq_kv_attention_ex(cache, batch, &view, Q, t, q_heads, q_stride, max_rows, scale, causal, O, o_stride, lse, workspace,
                               workspace_bytes, stream);
}

}  // extern "C"
