// C ABI of what surrounds attention in a step on the 4-bit key/value cache: its tables and the
// rotated append.  Host-side validation; see include/awq.h for the contract.
#include "kv_host.h"

#include <math.h>

using awq::kKvMaxCount;
using awq::kv_aligned;
using awq::kv_fail;

extern "C" {

awq_status awq_kv_append_rotated(const awq_kv_cache *cache, const awq_kv_batch *batch, const awq_kv_rotation *rotation,
                                 const void *Q, const void *K, const void *V, awq_dtype t, int64_t q_heads, int64_t q_stride,
                                 int64_t k_stride, int64_t v_stride, void *Q_out, int64_t q_out_stride, hipStream_t stream) {
    awq::KvCache c{};
    awq::KvBatch s{};
    awq_status e = awq::kv_check_copy(cache, batch, K, V, t, k_stride, v_stride, &c, &s);
    if (e != AWQ_OK) return e;
    if (!rotation) return kv_fail(AWQ_ERR_ARG, "rotation must be non-NULL");
    if (q_heads < 1 || q_heads > 65535) return kv_fail(AWQ_ERR_SHAPE, "q_heads must be in 1..65535 (got %lld)", static_cast<long long>(q_heads));
    if ((e = awq::kv_check_rows(Q, "Q", t, batch->rows, q_stride, q_heads * cache->dim)) != AWQ_OK) return e;
    if ((e = awq::kv_check_rows(Q_out, "Q_out", t, batch->rows, q_out_stride, q_heads * cache->dim)) != AWQ_OK) return e;
    if (Q_out == Q && q_out_stride != q_stride && batch->rows > 1)
        return kv_fail(AWQ_ERR_ARG, "in place, Q and Q_out must have one row stride");
    const awq_kv_rotation &r = *rotation;
    if (r.rot < 0 || r.rot > cache->dim || r.rot % 16 != 0)
        return kv_fail(AWQ_ERR_SHAPE, "rot must be a multiple of 16 in 0..%d (got %d)", cache->dim, r.rot);
    if (r.interleaved != 0 && r.interleaved != 1) return kv_fail(AWQ_ERR_ARG, "interleaved must be 0 or 1 (got %d)", r.interleaved);
    if (r.rot > 0 && (r.positions < 1 || r.positions > kKvMaxCount))
        return kv_fail(AWQ_ERR_SHAPE, "positions must be in 1..2^30 (got %lld)", static_cast<long long>(r.positions));
    if (r.rot > 0 && (!r.cos_sin || !kv_aligned(r.cos_sin, 16)))
        return kv_fail(AWQ_ERR_ARG, "cos_sin must be non-NULL, 16-byte aligned");
    if (!kv_aligned(r.q_weight, 16) || !kv_aligned(r.k_weight, 16))
        return kv_fail(AWQ_ERR_ARG, "q_weight and k_weight must be 16-byte aligned");
    if ((r.q_weight || r.k_weight) && (!(r.eps > 0.0) || !isfinite(r.eps)))
        return kv_fail(AWQ_ERR_ARG, "eps must be positive and finite (got %g)", r.eps);
    // (a launch has fewer than 2^32 threads: up to 2^31 for the keys' units, as kv_check says, and a wave to
    // 32, 16 or 8 query heads of a row; whole workgroups of both)
    const int64_t heads = 2048 / cache->dim, waves = batch->rows * ((q_heads + heads - 1) / heads);
    if (waves > (int64_t(1) << 25) - 64) return kv_fail(AWQ_ERR_SHAPE, "rows * q_heads too large for one call");
    if (s.T == 0) return AWQ_OK;
    // other workgroups read the queries, keys and values meanwhile
    const int64_t size = t == AWQ_F32 ? 4 : 2, q_width = q_heads * cache->dim * size, width = cache->heads * cache->dim * size;
    const awq::KvRowSpan out{Q_out, q_out_stride * size, q_width};
    if (Q_out != Q && awq::kv_rows_meet(out, {Q, q_stride * size, q_width}, s.T))
        return kv_fail(AWQ_ERR_ARG, "Q_out may be Q, but else must not share memory with it");
    const bool keys_first = awq::kv_rows_meet(out, {K, k_stride * size, width}, s.T) || awq::kv_rows_meet(out, {V, v_stride * size, width}, s.T);
    const awq::KvTurn turn{r.cos_sin, static_cast<int>(r.positions), r.rot, r.interleaved, r.q_weight, r.k_weight, r.eps, keys_first};
    return awq::kv_hip_status(awq::launch_kv_append_rotated(c, s, turn, Q, K, V, Q_out, t, static_cast<int>(q_heads), q_stride, k_stride,
                                                            v_stride, q_out_stride, stream),
                              "awq_kv_append_rotated launch");
}

awq_status awq_kv_tables(int page, int64_t batch, int64_t max_pages, const int32_t *kv_len, const int32_t *count,
                         const int32_t *free_pages, int64_t n_free, const int32_t *taken, int32_t *block_table, int64_t rows,
                         const awq_kv_step *step, hipStream_t stream) {
    return awq_kv_tables_ex(page, batch, max_pages, kv_len, count, free_pages, n_free, taken, block_table, rows, 0, step, stream);
}

awq_status awq_kv_tables_ex(int page, int64_t batch, int64_t max_pages, const int32_t *kv_len, const int32_t *count,
                            const int32_t *free_pages, int64_t n_free, const int32_t *taken, int32_t *block_table, int64_t rows,
                            int64_t n_pages, const awq_kv_step *step, hipStream_t stream) {
    awq::report_error(AWQ_OK, "");
    if (page < 16 || page > 256 || (page & (page - 1)) != 0)
        return kv_fail(AWQ_ERR_ARG, "page must be a power of two in 16..256 (got %d)", page);
    if (batch < 1 || batch > (int64_t(1) << 21)) return kv_fail(AWQ_ERR_SHAPE, "batch must be in 1..2^21 (got %lld)", static_cast<long long>(batch));
    if (max_pages < 1 || max_pages > kKvMaxCount || max_pages * page > kKvMaxCount)
        return kv_fail(AWQ_ERR_SHAPE, "max_pages must be >= 1 and hold at most 2^30 positions");
    if (rows < 0 || rows > kKvMaxCount) return kv_fail(AWQ_ERR_SHAPE, "rows must be in 0..2^30 (got %lld)", static_cast<long long>(rows));
    if (n_free < 0 || n_free > INT32_MAX) return kv_fail(AWQ_ERR_SHAPE, "n_free must be in 0..2^31-1 (got %lld)", static_cast<long long>(n_free));
    if (!kv_len || !count || !block_table || (n_free > 0 && !free_pages))
        return kv_fail(AWQ_ERR_ARG, "kv_len, count, free_pages and block_table must be non-NULL");
    if (!step || !step->kv_len || !step->row_start || !step->taken)
        return kv_fail(AWQ_ERR_ARG, "step and its kv_len, row_start and taken must be non-NULL");
    if (n_pages < 0 || n_pages > INT32_MAX)
        return kv_fail(AWQ_ERR_SHAPE, "n_pages must be in 0..2^31-1 (got %lld)", static_cast<long long>(n_pages));
    struct Part {
        const void *p;
        int64_t n;   // elements
        int size;
    };
    const Part in[] = {{kv_len, batch, 4}, {count, batch, 4}, {free_pages, n_free, 4}, {taken, 1, 4}};
    const Part out[] = {{step->kv_len, batch, 4}, {step->row_start, batch + 1, 4}, {step->taken, 1, 4}, {step->position, rows, 4},
                        {step->slot, rows, 8}, {block_table, batch * max_pages, 4}};
    for (const Part &x : in)
        if (!kv_aligned(x.p, 4)) return kv_fail(AWQ_ERR_ARG, "kv_len, count, free_pages and taken must be 4-byte aligned");
    for (const Part &y : out)
        if (!kv_aligned(y.p, y.size)) return kv_fail(AWQ_ERR_ARG, "outputs must be aligned to their elements");
    // workgroups read the inputs while others write the outputs
    auto meet = [](const Part &x, const Part &y) {
        const uintptr_t x0 = reinterpret_cast<uintptr_t>(x.p), y0 = reinterpret_cast<uintptr_t>(y.p);
        return x0 && y0 && x.n > 0 && y.n > 0 && x0 < y0 + y.n * y.size && y0 < x0 + x.n * x.size;
    };
    for (const Part &y : out) {
        for (const Part &x : in)
            if (meet(x, y)) return kv_fail(AWQ_ERR_ARG, "no output may share memory with an input");
        for (const Part *x = out; x != &y; ++x)
            if (meet(*x, y)) return kv_fail(AWQ_ERR_ARG, "no output may share memory with another");
    }
    awq::KvTables a{};
    a.kv_len = kv_len, a.count = count, a.free_pages = free_pages, a.taken = taken;
    a.n_free = n_free, a.T = step->position || step->slot ? rows : 0;
    a.table = block_table, a.new_len = step->kv_len, a.row_start = step->row_start, a.new_taken = step->taken;
    a.position = step->position, a.slot = step->slot;
    a.n_pages = n_pages > 0 ? n_pages : int64_t(1) << 31;
    a.B = static_cast<int>(batch), a.max_pages = static_cast<int>(max_pages);
    while ((1 << a.page_shift) < page) ++a.page_shift;
    return awq::kv_hip_status(awq::launch_kv_tables(a, stream), "awq_kv_tables launch");
}

}  // extern "C"
