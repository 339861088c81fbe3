// C ABI of the 4-bit key/value cache: host-side validation, workspace layout
// and the choice of launches.  See include/awq.h for the contract.
#include "awq.h"  // include/awq.h (on the -I path)

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "kv_internal.h"

namespace {

awq_status fail(awq_status code, const char *fmt, ...) {
    char msg[384];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return static_cast<awq_status>(awq::report_error(code, msg));
}

awq_status hip_status(hipError_t e, const char *what) {
    if (e == hipSuccess) return AWQ_OK;
    return fail(AWQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

constexpr int64_t kMaxCount = int64_t(1) << 30;   // rows, columns, units and tiles stay int32
// A launch has fewer than 2^32 threads: dim/2 to a unit of the copy kernels, and on the
// wide path of the attention at most 512 to an item and to 256 of its columns.
constexpr int64_t kMaxUnits = int64_t(1) << 25;   // (at dim 128)
constexpr int64_t kMaxItems = int64_t(1) << 21;   // batch * heads

// The sizes of a cache: 0 or the bytes of one (page, head).
int64_t block_bytes(int page, int64_t heads, int dim, int group) {
    if (dim != 64 && dim != 128 && dim != 256) {
        fail(AWQ_ERR_SHAPE, "dim must be 64, 128 or 256 (got %d)", dim);
        return 0;
    }
    if ((group != 32 && group != 64 && group != 128) || group > dim) {
        fail(AWQ_ERR_ARG, "group must be 32, 64 or 128 and at most dim (got %d)", group);
        return 0;
    }
    if (page < 16 || page > 256 || (page & (page - 1)) != 0) {
        fail(AWQ_ERR_ARG, "page must be a power of two in 16..256 (got %d)", page);
        return 0;
    }
    if (heads < 1 || heads > 65535) {
        fail(AWQ_ERR_SHAPE, "heads must be in 1..65535 (got %lld)", static_cast<long long>(heads));
        return 0;
    }
    return static_cast<int64_t>(page) * dim + 8ll * page * (dim / group);
}

awq_status check(const awq_kv_cache *cache, const awq_kv_batch *batch, awq::KvCache *c, awq::KvBatch *s,
                 bool sizes_only = false) {
    if (!cache || !batch) return fail(AWQ_ERR_ARG, "cache and batch must be non-NULL");
    const int64_t block = block_bytes(cache->page, cache->heads, cache->dim, cache->group);
    if (block == 0) return cache->dim != 64 && cache->dim != 128 && cache->dim != 256 ? AWQ_ERR_SHAPE
                           : cache->heads < 1 || cache->heads > 65535                ? AWQ_ERR_SHAPE
                                                                                      : AWQ_ERR_ARG;
    if (batch->batch < 1 || batch->batch > kMaxCount) return fail(AWQ_ERR_SHAPE, "batch must be >= 1");
    if (batch->rows < 0 || batch->rows > kMaxCount) return fail(AWQ_ERR_SHAPE, "rows must be >= 0");
    if (batch->max_pages < 1 || batch->max_pages > kMaxCount || batch->max_pages * cache->page > kMaxCount)
        return fail(AWQ_ERR_SHAPE, "max_pages must be >= 1 and hold at most 2^30 positions");
    if (!batch->row_start && batch->rows % batch->batch != 0)
        return fail(AWQ_ERR_SHAPE, "without row_start, rows (%lld) must be a multiple of batch (%lld)",
                    static_cast<long long>(batch->rows), static_cast<long long>(batch->batch));
    const int64_t tiles = (batch->max_pages * cache->page + awq::kKvTile - 1) / awq::kKvTile;
    // units of the copy kernels, and tiles of the attention's line
    if ((batch->rows / 4 + 2 * batch->batch) * cache->heads > kMaxUnits * 128 / cache->dim ||
        batch->batch * cache->heads > kMaxItems ||
        batch->batch * cache->heads * (tiles + awq::kKvItemCost) > kMaxCount)
        return fail(AWQ_ERR_SHAPE, "batch * heads * max_pages or rows * heads too large for one call");
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
    if (cache->n_pages < 1 || cache->n_pages > INT32_MAX) return fail(AWQ_ERR_SHAPE, "n_pages must be in 1..2^31-1");
    if (cache->page_stride < cache->heads * block || cache->page_stride % 16 != 0)
        return fail(AWQ_ERR_SHAPE, "page_stride must be a multiple of 16 and at least %lld bytes (got %lld)",
                    static_cast<long long>(cache->heads * block), static_cast<long long>(cache->page_stride));
    if (!cache->pages || !aligned(cache->pages, 16)) return fail(AWQ_ERR_ARG, "pages must be non-NULL, 16-byte aligned");
    if (!batch->kv_len || !batch->block_table) return fail(AWQ_ERR_ARG, "kv_len and block_table must be non-NULL");
    if (!aligned(batch->kv_len, 4) || !aligned(batch->block_table, 4) || !aligned(batch->row_start, 4))
        return fail(AWQ_ERR_ARG, "row_start, kv_len and block_table must be 4-byte aligned");
    return AWQ_OK;
}

bool wide_type(awq_dtype t) { return t == AWQ_F32 || t == AWQ_BF16 || t == AWQ_F16; }

awq_status check_rows(const void *p, const char *name, awq_dtype t, int64_t rows, int64_t stride, int64_t least) {
    if (rows > 0 && !p) return fail(AWQ_ERR_ARG, "%s must be non-NULL", name);
    if (!aligned(p, 16)) return fail(AWQ_ERR_ARG, "%s must be 16-byte aligned", name);
    const int64_t size = t == AWQ_F32 ? 4 : 2;
    if (stride < least || stride > kMaxCount || stride * size % 16 != 0)
        return fail(AWQ_ERR_SHAPE, "the row stride of %s must be at least %lld elements and a multiple of 16 bytes "
                    "(got %lld)", name, static_cast<long long>(least), static_cast<long long>(stride));
    return AWQ_OK;
}

awq_status copy_checks(const awq_kv_cache *cache, const awq_kv_batch *batch, const void *K, const void *V, awq_dtype t,
                       int64_t k_stride, int64_t v_stride, awq::KvCache *c, awq::KvBatch *s) {
    awq::report_error(AWQ_OK, "");
    awq_status e = check(cache, batch, c, s);
    if (e != AWQ_OK) return e;
    if (!wide_type(t)) return fail(AWQ_ERR_DTYPE, "unsupported dtype %d", static_cast<int>(t));
    const int64_t least = cache->heads * cache->dim;
    if ((e = check_rows(K, "K", t, batch->rows, k_stride, least)) != AWQ_OK) return e;
    return check_rows(V, "V", t, batch->rows, v_stride, least);
}

// The launches of one attention call and its workspace (byte offsets).
struct Plan {
    bool split, wide, merge, line, wide_merge;
    int snap, tiles_col, split_cols, workers, units, wide_workers;
    size_t items, part_ml, part, wide_items, wide_ml, wide_part, total;
};

constexpr int kSimds = 4 * awq::kKvCus;

awq_status plan(const awq::KvCache &c, const awq::KvBatch &s, int64_t q_heads, int64_t max_rows, Plan *p) {
    if (q_heads < 1 || q_heads > 65535 || q_heads % c.heads != 0)
        return fail(AWQ_ERR_SHAPE, "q_heads (%lld) must be a multiple of the cache's heads (%d)",
                    static_cast<long long>(q_heads), c.heads);
    if (max_rows < 0) return fail(AWQ_ERR_SHAPE, "max_rows must be >= 0");
    if (static_cast<int64_t>(s.T) * q_heads > kMaxCount) return fail(AWQ_ERR_SHAPE, "rows * q_heads too large for one call");
    const int64_t per = q_heads / c.heads;
    const int64_t most = s.row_start ? (max_rows == 0 || max_rows > s.T ? s.T : max_rows) : s.even;
    const int64_t cols = most * per, limit = awq::kv_split_cols(c.dim);
    const int64_t tiles = (static_cast<int64_t>(s.max_pages) * (1 << c.page_shift) + awq::kKvTile - 1) / awq::kKvTile;
    *p = Plan{};
    p->wide = cols > limit;
    // Where the wide path runs, the split path is for its single tokens.
    const int64_t need = p->wide ? per : cols;
    p->split = need <= limit && (!p->wide || s.row_start);
    p->tiles_col = need <= 16 ? 1 : need <= 32 ? 2 : 4;
    // What a sequence's columns are compared with on the device is what the workspace holds for
    // each piece: one with more rows than max_rows is left out, not kept in too small a place.
    p->split_cols = p->split ? static_cast<int>(p->wide ? 16 * p->tiles_col : need) : 0;
    const int64_t line = s.B * static_cast<int64_t>(c.heads) * (tiles + awq::kKvItemCost);
    const int64_t useful = (line + awq::kKvMinShare - 1) / awq::kKvMinShare;
    const int64_t fill = kSimds * awq::kv_split_waves(c.dim, p->tiles_col);
    p->workers = static_cast<int>(useful < fill ? useful : fill);
    p->snap = static_cast<int>(tiles <= awq::kKvWhole ? tiles : awq::kKvSnap);
    p->merge = p->split && tiles > 2 * p->snap + 1;   // shorter items are never cut
    const int64_t wide = awq::kv_wide_cols(c.dim);
    p->units = static_cast<int>(s.row_start ? s.T * per / wide + s.B : s.B * ((s.even * per + wide - 1) / wide));
    const int64_t groups = static_cast<int64_t>(p->units) * c.heads;
    const int64_t wide_tiles = (static_cast<int64_t>(s.max_pages) * (1 << c.page_shift) - 1) / awq::kv_wide_tile(c.dim) + 1;
    const int64_t wide_line = groups * (wide_tiles + awq::kKvWideCost);
    p->line = p->wide && groups < awq::kKvLineUnits && wide_line <= kMaxCount;
    const int64_t wide_useful = (wide_line + awq::kKvWideMinShare - 1) / awq::kKvWideMinShare;
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
        p->items = take(static_cast<size_t>(s.B) * c.heads * 8);
        p->part_ml = take(n * 8);
        p->part = take(n * c.dim * 4);
    }
    if (p->wide_merge) {
        const size_t n = static_cast<size_t>(p->wide_workers) * 2 * wide;
        p->wide_items = take(static_cast<size_t>(groups) * 8);
        p->wide_ml = take(n * 8);
        p->wide_part = take(n * c.dim * 4);
    }
    p->total = at;
    return AWQ_OK;
}

}  // namespace

extern "C" {

size_t awq_kv_page_size(int page, int64_t heads, int dim, int group) {
    awq::report_error(AWQ_OK, "");
    return static_cast<size_t>(block_bytes(page, heads, dim, group) * heads);
}

awq_status awq_kv_append(const awq_kv_cache *cache, const awq_kv_batch *batch, const void *K, const void *V,
                         awq_dtype t, int64_t k_stride, int64_t v_stride, hipStream_t stream) {
    awq::KvCache c{};
    awq::KvBatch s{};
    const awq_status e = copy_checks(cache, batch, K, V, t, k_stride, v_stride, &c, &s);
    if (e != AWQ_OK || s.T == 0) return e;
    return hip_status(awq::launch_kv_append(c, s, K, V, t, k_stride, v_stride, stream), "awq_kv_append launch");
}

awq_status awq_kv_read(const awq_kv_cache *cache, const awq_kv_batch *batch, void *K, void *V, awq_dtype t,
                       int64_t k_stride, int64_t v_stride, hipStream_t stream) {
    awq::KvCache c{};
    awq::KvBatch s{};
    const awq_status e = copy_checks(cache, batch, K, V, t, k_stride, v_stride, &c, &s);
    if (e != AWQ_OK || s.T == 0) return e;
    return hip_status(awq::launch_kv_read(c, s, K, V, t, k_stride, v_stride, stream), "awq_kv_read launch");
}

size_t awq_kv_attention_workspace_size(const awq_kv_cache *cache, const awq_kv_batch *batch, int64_t q_heads,
                                       int64_t max_rows) {
    awq::report_error(AWQ_OK, "");
    awq::KvCache c{};
    awq::KvBatch s{};
    Plan p{};
    if (check(cache, batch, &c, &s, true) != AWQ_OK || plan(c, s, q_heads, max_rows, &p) != AWQ_OK) return 0;
    return p.total;
}

awq_status awq_kv_attention(const awq_kv_cache *cache, const awq_kv_batch *batch, const void *Q, awq_dtype t,
                            int64_t q_heads, int64_t q_stride, int64_t max_rows, float scale, int causal,
                            int64_t window, void *O, int64_t o_stride, float *lse, void *workspace,
                            size_t workspace_bytes, hipStream_t stream) {
    awq::report_error(AWQ_OK, "");
    awq::KvAttend a{};
    Plan p{};
    awq_status e = check(cache, batch, &a.c, &a.s);
    if (e != AWQ_OK) return e;
    if (t != AWQ_BF16 && t != AWQ_F16) return fail(AWQ_ERR_DTYPE, "Q must be AWQ_BF16 or AWQ_F16 (got %d)", static_cast<int>(t));
    if ((e = plan(a.c, a.s, q_heads, max_rows, &p)) != AWQ_OK) return e;
    const int64_t least = q_heads * cache->dim;
    if ((e = check_rows(Q, "Q", t, batch->rows, q_stride, least)) != AWQ_OK) return e;
    if ((e = check_rows(O, "O", t, batch->rows, o_stride, least)) != AWQ_OK) return e;
    if (!aligned(lse, 4)) return fail(AWQ_ERR_ARG, "lse must be 4-byte aligned");
    if (!(scale > 0.0f) || !isfinite(scale)) return fail(AWQ_ERR_ARG, "scale must be positive and finite (got %g)", scale);
    if (causal != 0 && causal != 1) return fail(AWQ_ERR_ARG, "causal must be 0 or 1 (got %d)", causal);
    if (window < 0) return fail(AWQ_ERR_ARG, "window must be >= 0 (0: none)");
    if (window > 0 && !causal) return fail(AWQ_ERR_ARG, "a window needs causal = 1");
    if (batch->rows == 0) return AWQ_OK;
    if (p.total > 0) {
        if (!workspace) return fail(AWQ_ERR_WORKSPACE, "workspace is NULL (need %zu bytes)", p.total);
        if (!aligned(workspace, 16)) return fail(AWQ_ERR_WORKSPACE, "workspace must be 16-byte aligned");
        if (workspace_bytes < p.total)
            return fail(AWQ_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", workspace_bytes, p.total);
    }
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
    if (p.merge) {
        a.items = reinterpret_cast<int2 *>(ws + p.items);
        a.part_ml = reinterpret_cast<float *>(ws + p.part_ml);
        a.part = reinterpret_cast<float *>(ws + p.part);
    }
    if (p.wide_merge) {
        a.wide_items = reinterpret_cast<int2 *>(ws + p.wide_items);
        a.wide_ml = reinterpret_cast<float *>(ws + p.wide_ml);
        a.wide_part = reinterpret_cast<float *>(ws + p.wide_part);
    }
    hipError_t h;
    if (a.c.dim == 64)
        h = awq::launch_kv_attend_64(a, t, p.split, p.wide, p.merge, stream);
    else if (a.c.dim == 128)
        h = awq::launch_kv_attend_128(a, t, p.split, p.wide, p.merge, stream);
    else
        h = awq::launch_kv_attend_256(a, t, p.split, p.wide, p.merge, stream);
    return hip_status(h, "awq_kv_attention launch");
}

}  // extern "C"
