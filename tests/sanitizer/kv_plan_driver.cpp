// Walks the split path's line on the host, with the kernels' own arithmetic, over
// the arguments that awq_kv_attention hands to its launches: every piece of every
// worker has to lie in its own place of the workspace, whatever the rows on the
// device are, and the pieces of an item have to make up the item.  The launches are
// replaced by the walk; nothing reaches a device.
#include "awq.h"

#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "kv_internal.h"

#define CHECK(x)                                                        \
    do {                                                                \
        if (!(x)) {                                                     \
            std::printf("FAILED %s:%d: %s\n", __FILE__, __LINE__, #x);  \
            std::exit(1);                                               \
        }                                                               \
    } while (0)

static size_t workspace_bytes;
static unsigned char *const workspace = reinterpret_cast<unsigned char *>(uintptr_t(1) << 40);
static long long kept, left_out, walks;

static void walk(const awq::KvAttend &a, bool merge) {
    struct Item { int b, head, n, tiles, begin, end, covered, first, pieces; };
    std::vector<Item> items;
    int total = 0;
    for (int b = 0; b < a.s.B; ++b) {
        int r0, n, len;
        const int tiles = awq::kv_item_tiles(a, b, r0, n, len);
        if (tiles == 0 && n > 0) ++left_out;
        for (int h = 0; h < a.c.heads && tiles > 0; ++h) {
            items.push_back({b, h, n, tiles, total, total + tiles + awq::kKvItemCost, 0, -1, 0});
            total = items.back().end;
        }
    }
    ++walks;
    if (total == 0) return;
    const int workers = awq::kv_workers(a, total);
    CHECK(workers >= 1 && workers <= a.workers);
    CHECK(awq::kv_share(0, total, workers) == 0 && awq::kv_share(workers, total, workers) == total);
    const float *const part_end = !merge ? nullptr : a.part + int64_t(a.workers) * 2 * a.split_cols * a.c.dim;
    if (merge) {
        CHECK(reinterpret_cast<unsigned char *>(a.items) >= workspace);
        CHECK(reinterpret_cast<unsigned char *>(a.items + int64_t(a.s.B) * a.c.heads) <= reinterpret_cast<unsigned char *>(a.part_ml));
        CHECK(reinterpret_cast<const unsigned char *>(part_end) <= workspace + workspace_bytes);
    } else {
        CHECK(!a.items && !a.part && !a.part_ml);
    }
    std::vector<int> used(merge ? size_t(a.workers) * 2 * a.split_cols : 0, -1);
    size_t i = 0;
    for (int w = 0; w < workers; ++w) {
        const int x0 = awq::kv_share(w, total, workers), x1 = awq::kv_share(w + 1, total, workers);
        while (items[i].end <= x0) ++i;
        for (size_t k = i; k < items.size() && items[k].begin < x1; ++k) {
            Item &it = items[k];
            const int t0 = x0 <= it.begin ? 0 : awq::kv_cut(a, it.begin, it.tiles, x0);
            const int t1 = x1 >= it.end ? it.tiles : awq::kv_cut(a, it.begin, it.tiles, x1);
            if (t0 >= t1) continue;
            CHECK(t0 == it.covered);   // in order, without gaps
            it.covered = t1;
            if (t0 == 0 && t1 == it.tiles) continue;
            CHECK(merge);
            const int64_t at = awq::kv_piece(a, w, t0 == 0), cols = int64_t(it.n) * a.per;   // what the kernel keeps
            const float *const out = a.part + at * a.c.dim, *const ml = a.part_ml + 2 * at;
            CHECK(out + cols * a.c.dim <= part_end && ml + 2 * cols <= a.part);
            for (int64_t c = at; c < at + cols; ++c) {
                CHECK(used[c] == -1);
                used[c] = w;
            }
            if (it.first < 0) it.first = w;
            ++it.pieces;
            ++kept;
        }
    }
    for (const Item &it : items) {
        CHECK(it.covered == it.tiles);
        if (it.first < 0) continue;
        const int last = static_cast<int>((static_cast<int64_t>(it.end - a.snap) * workers + total - 1) / total) - 1;
        CHECK(it.pieces == last - it.first + 1);   // as the kernel tells the join
    }
}

namespace awq {
static hipError_t seen(const KvAttend &a, bool split, bool merge) {
    if (split) walk(a, merge);
    return hipSuccess;
}
hipError_t launch_kv_attend_64(const KvAttend &a, int, bool s, bool, bool m, hipStream_t) { return seen(a, s, m); }
hipError_t launch_kv_attend_128(const KvAttend &a, int, bool s, bool, bool m, hipStream_t) { return seen(a, s, m); }
hipError_t launch_kv_attend_256(const KvAttend &a, int, bool s, bool, bool m, hipStream_t) { return seen(a, s, m); }
hipError_t launch_kv_append(const KvCache &, const KvBatch &, const void *, const void *, int, int64_t, int64_t, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_kv_read(const KvCache &, const KvBatch &, void *, void *, int, int64_t, int64_t, hipStream_t) {
    return hipSuccess;
}
}  // namespace awq

int main() {
    std::mt19937 rng(1);
    auto pick = [&](std::initializer_list<int> v) { return *(v.begin() + rng() % v.size()); };
    for (int round = 0; round < 4000; ++round) {
        awq_kv_cache c{};
        c.pages = workspace, c.n_pages = 1 << 20, c.dim = pick({64, 128, 256}), c.group = pick({32, 64}), c.page = pick({16, 64, 256});
        c.heads = pick({1, 2, 5, 8});
        c.page_stride = static_cast<int64_t>(awq_kv_page_size(c.page, c.heads, c.dim, c.group));
        const int batch = pick({1, 2, 3, 17, 64, 65, 130}), per = pick({1, 1, 2, 3, 4, 8, 16, 32, 71});
        const int span = pick({1, 6, 7, 40, 400}) * 64 / c.page + 1;
        // max_rows below, at and above what the sequences have: rows on the device can change under a captured graph
        const int max_rows = pick({1, 1, 1, 2, 3, 5, 8, 16, 0}), most = pick({1, 2, 4, 16, 17, 64, 200});
        std::vector<int32_t> start(batch + 1), len(batch);
        for (int b = 0; b < batch; ++b) {
            const int n = rng() % 3 == 0 ? static_cast<int>(rng() % (most + 1)) : rng() % 8 == 0 ? 0 : 1;
            start[b + 1] = start[b] + n;
            len[b] = static_cast<int32_t>(rng() % 4 == 0 ? span * c.page : rng() % (span * c.page + 40));
        }
        awq_kv_batch s{};
        s.rows = start[batch] + rng() % 3, s.batch = batch, s.max_pages = span, s.kv_len = len.data(), s.block_table = len.data();
        s.row_start = start.data();
        if (round % 7 == 0) {   // the same rows for each
            s.row_start = nullptr;
            s.rows = int64_t(batch) * pick({1, 2, 5});
        } else if (round % 7 == 1) {   // and nonsense, which the kernels bound
            for (auto &x : start) x = static_cast<int32_t>(rng());
            for (auto &x : len) x = static_cast<int32_t>(rng());
        }
        const int64_t q_heads = per * c.heads;
        workspace_bytes = awq_kv_attention_workspace_size(&c, &s, q_heads, max_rows);
        const int window = pick({0, 0, 1, 33, 1000});
        const awq_status e = awq_kv_attention(&c, &s, workspace, AWQ_BF16, q_heads, q_heads * c.dim, max_rows, 1.0f, 1, window,
                                              workspace, q_heads * c.dim, nullptr, workspace, workspace_bytes, nullptr);
        if (e != AWQ_OK) std::printf("%s\n", awq_last_error());
        CHECK(e == AWQ_OK);
    }
    CHECK(kept > 10000 && left_out > 1000);
    std::printf("%lld walks, %lld pieces in their places, %lld sequences left out\n", walks, kept, left_out);
    return 0;
}
