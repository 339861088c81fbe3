// The wide path's schedule of a tile's unpacking, slot by slot, for every head
// dimension: each part of each value piece once and in order, each piece's pairs
// read before its first part and after the last of the piece before, no piece that does
// not exist, and the next loads behind the last part.
#include <cstdio>
#include <cstdlib>

#include "kv_attend.h"

#define CHECK(x)                                                                       \
    do {                                                                               \
        if (!(x)) {                                                                    \
            std::printf("FAILED %s:%d (dim %d): %s\n", __FILE__, __LINE__, D, #x);     \
            std::exit(1);                                                              \
        }                                                                              \
    } while (0)

template <int D>
static void schedule() {
    typedef awq::KvWideLoad<D, 1, awq::kv_wide_threads(D)> Load;
    int part = 0, pairs = 0;
    for (int slot = 0; slot < Load::kSlots; ++slot) {
        const int p = Load::part_at(slot), q = Load::pairs_at(slot);   // in a slot, the part comes first
        CHECK(p >= -1 && p < 4 * Load::VI && q >= -1 && q < Load::VI);
        if (p >= 0) {
            CHECK(slot > Load::KW && p == part && pairs == part / 4 + 1);
            ++part;
        }
        if (q >= 0) {
            CHECK(q == pairs && part == 4 * q);
            ++pairs;
        }
        if (slot == Load::kLoad) CHECK(part == 4 * Load::VI);
    }
    CHECK(part == 4 * Load::VI && pairs == Load::VI && Load::kLoad < Load::kSlots && Load::KW < Load::kSlots);
}

int main() {
    schedule<64>();
    schedule<128>();
    schedule<256>();
    std::printf("schedules hold\n");
    return 0;
}
