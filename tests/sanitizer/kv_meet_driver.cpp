// kv_rows_meet against a map of every byte.
#include "kv_host.h"

#include <cstdio>
#include <cstdlib>
#include <vector>

int main() {
    long long checked = 0, met = 0, between = 0;
    const int64_t strides[] = {2, 4, 6, 10, 12, 18};
    for (int64_t rows = 0; rows <= 5; ++rows)
        for (int64_t xs : strides)
            for (int64_t ys : strides)
                for (int64_t xw : {int64_t(2), int64_t(4), int64_t(6), xs})
                    for (int64_t yw : {int64_t(2), int64_t(4), int64_t(6), ys})
                        for (int64_t at = 0; at < 200; at += 2) {
                            if (xw > xs || yw > ys) continue;
                            std::vector<bool> used(400);
                            for (int64_t r = 0; r < rows; ++r)
                                for (int64_t i = 0; i < xw; ++i) used[80 + r * xs + i] = true;
                            bool shared = false;
                            for (int64_t r = 0; r < rows; ++r)
                                for (int64_t i = 0; i < yw; ++i) shared |= used[at + r * ys + i];
                            const char *base = reinterpret_cast<const char *>(uintptr_t(1) << 40);
                            const awq::KvRowSpan x{base + 80, xs, xw}, y{base + at, ys, yw};
                            const bool said = awq::kv_rows_meet(x, y, rows);
                            if (shared != said || said != awq::kv_rows_meet(y, x, rows)) {
                                std::printf("FAILED rows %lld strides %lld %lld widths %lld %lld at %lld: %d, %d said\n", (long long)rows,
                                            (long long)xs, (long long)ys, (long long)xw, (long long)yw, (long long)at - 80, shared, said);
                                return 1;
                            }
                            ++checked, met += shared, between += !shared && xs != ys && at > 80 && at < 80 + rows * xs;
                        }
    // ends of the types that the checks let through
    const int64_t most = int64_t(1) << 30;
    const awq::KvRowSpan x{reinterpret_cast<void *>(uintptr_t(16)), most * 4, most * 4}, y{reinterpret_cast<void *>(~uintptr_t(0) - 15), 16, 16};
    if (awq::kv_rows_meet(x, {reinterpret_cast<void *>(uintptr_t(1) << 62), 16, 16}, 1) || !awq::kv_rows_meet(x, x, most) ||
        awq::kv_rows_meet(x, y, 1)) return 1;
    // many rows that pass between each other's
    const awq::KvRowSpan even{reinterpret_cast<void *>(uintptr_t(1) << 40), 64, 16}, odd{reinterpret_cast<void *>((uintptr_t(1) << 40) + 32), 192, 16};
    if (awq::kv_rows_meet(even, odd, 1 << 20) || awq::kv_rows_meet(odd, even, 1 << 20)) return 1;
    std::printf("%lld checked, %lld met, %lld rows of two strides between each other\n", checked, met, between);
    return met > 10000 && between > 1000 ? 0 : 1;
}
