// Attention over the 4-bit key/value cache, head dimension 128 (kv_attend.h).
#include "kv_attend.h"

namespace awq {

hipError_t launch_kv_attend_128(const KvAttend &a, int type, bool run_split, bool run_wide, bool merge,
                               hipStream_t st) {
    if (a.c.group == 32) return kv_attend_group<128, 4>(a, type, run_split, run_wide, merge, st);
    if (a.c.group == 64) return kv_attend_group<128, 2>(a, type, run_split, run_wide, merge, st);
    if (a.c.group == 128) return kv_attend_group<128, 1>(a, type, run_split, run_wide, merge, st);
    return hipErrorInvalidValue;
}

}  // namespace awq
