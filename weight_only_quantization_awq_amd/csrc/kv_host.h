// Host side of the key/value cache's entry points: checks that awq_kv.hip and
// awq_kv_step.hip share.  Each sets awq_last_error() where it refuses.
#pragma once

#include "awq.h"  // include/awq.h (on the -I path)

#include "kv_internal.h"

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

// kv_check and the keys and values of a call that writes or reads them.
awq_status kv_check_copy(const awq_kv_cache *cache, const awq_kv_batch *batch, const void *K, const void *V, awq_dtype t,
                         int64_t k_stride, int64_t v_stride, KvCache *c, KvBatch *s);

}  // namespace awq
