// Host side of the key/value cache's entry points: checks that awq_kv.hip and
// awq_kv_step.hip share.  Each sets awq_last_error() where it refuses.
#pragma once

#include "awq.h"  // include/awq.h (on the -I path)

#include "kv_internal.h"

#include <numeric>

namespace awq {

constexpr int64_t kKvMaxCount = int64_t(1) << 30;   // rows, columns, units and tiles stay int32

inline bool kv_aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

awq_status kv_fail(awq_status code, const char *fmt, ...);
awq_status kv_hip_status(hipError_t e, const char *what);

// Bytes of one page; 0 where the sizes are refused.
size_t kv_page_bytes(int page, int64_t heads, int dim, int group);

// A call's cache and sequences, as the kernels take them.  sizes_only: without the pointers.
awq_status kv_check(const awq_kv_cache *cache, const awq_kv_batch *batch, KvCache *c, KvBatch *s, bool sizes_only = false);

bool kv_wide_type(awq_dtype t);

// A tensor of `rows` rows of at least `least` elements, `stride` elements apart.
awq_status kv_check_rows(const void *p, const char *name, awq_dtype t, int64_t rows, int64_t stride, int64_t least);

// A tensor of rows, in bytes: `stride` apart, `width` of each in use.
struct KvRowSpan {
    const void *p;
    int64_t stride, width;
};
// Whether two of them share memory.  (Row by row only where the strides differ and their greatest
// common divisor does not settle it, inside the memory that both extend over.)
inline bool kv_rows_meet(const KvRowSpan &x, const KvRowSpan &y, int64_t rows) {
    const uint64_t x0 = reinterpret_cast<uintptr_t>(x.p), y0 = reinterpret_cast<uintptr_t>(y.p);
    if (rows < 1 || x0 >= y0 + (rows - 1) * y.stride + y.width || y0 >= x0 + (rows - 1) * x.stride + x.width) return false;
    if (rows == 1) return true;
    const int64_t each = std::gcd(x.stride, y.stride), ahead = static_cast<int64_t>(y0 - x0);   // (they meet, so it fits)
    const int64_t from = (ahead % each + each) % each;   // y's first byte behind a row of x, in the finest order of both
    if (from >= x.width && each - from >= y.width) return false;
    if (x.stride == y.stride) return true;
    const int64_t first = ahead - x.width < 0 ? 0 : (ahead - x.width) / x.stride;
    for (int64_t i = first; i < rows; ++i) {
        const int64_t at = i * x.stride - ahead;   // behind y's first byte
        if (at >= (rows - 1) * y.stride + y.width) return false;
        if (at < 0 ? at + x.width > 0 : at / y.stride < rows && at % y.stride < y.width) return true;
        const int64_t next = at < 0 ? 0 : at / y.stride + 1;   // the first row of y that begins behind it
        if (next < rows && next * y.stride < at + x.width) return true;
    }
    return false;
}

// kv_check and the keys and values of a call that writes or reads them.
awq_status kv_check_copy(const awq_kv_cache *cache, const awq_kv_batch *batch, const void *K, const void *V, awq_dtype t,
                         int64_t k_stride, int64_t v_stride, KvCache *c, KvBatch *s);

}  // namespace awq
