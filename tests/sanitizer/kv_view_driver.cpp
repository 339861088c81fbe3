// Walks the split path's line of calls with sinks and with a shared prefix on the host, with
// the kernels' own arithmetic, over the arguments that awq_kv_attention_ex hands to its launches:
// every piece in a place of its own inside the workspace, the pieces of an item making it up, the
// prefix's items among them, and every part of the workspace apart from the others.  Then
// the entry points of a step's tables and of the rotated append, with arguments at the ends of their
// types.  The launches are replaced by the walk; nothing reaches a device.
#include "awq.h"

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <limits>
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
static long long kept, prefix_pieces, sink_items, walks, launched, lines_apart;

struct Range { const unsigned char *from, *to; };
static std::vector<Range> ranges;
static void own(const void *p, int64_t bytes) {
    const unsigned char *q = static_cast<const unsigned char *>(p);
    CHECK(q >= workspace && q + bytes <= workspace + workspace_bytes && (reinterpret_cast<uintptr_t>(q) & 15) == 0);
    for (const Range &r : ranges) CHECK(q + bytes <= r.from || q >= r.to);
    ranges.push_back({q, q + bytes});
}

template <typename A>
static void walk(const A &a, bool merge) {
    struct Item { int b, head, n, tiles, begin, end, covered, first, pieces; };
    std::vector<Item> items;
    int total = 0;
    const int common = awq::kv_common(a);
    for (int b = 0; b < awq::kv_count(a); ++b) {
        int r0, n, len;
        const int tiles = awq::kv_item_tiles(a, b, r0, n, len, common);
        CHECK(r0 >= 0 && n >= 0 && r0 + n <= a.s.T && len >= 0);
        const int before = awq::kv_is_prefix(a, b) ? 0 : common, first = awq::kv_first_token(a, len, n, before);
        CHECK(first >= 0 && first <= len && awq::kv_lowest(a, len, n, before) >= first);
        const int sinks = awq::kv_sink_tiles(a, first, awq::kKvTile);
        CHECK(sinks >= 0 && sinks * awq::kKvTile <= first && (tiles == 0 || tiles > sinks));
        sink_items += sinks > 0;
        for (int h = 0; h < a.c.heads && tiles > 0; ++h) {
            items.push_back({b, h, n, tiles, total, total + tiles + awq::kKvItemCost, 0, -1, 0});
            total = items.back().end;
        }
    }
    ++walks;
    if (total == 0) return;
    const int workers = awq::kv_workers(a, total);
    CHECK(workers >= 1 && workers <= a.workers);
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
            CHECK(t0 == it.covered);
            it.covered = t1;
            if (t0 == 0 && t1 == it.tiles) continue;
            CHECK(merge);
            const int64_t at = awq::kv_piece(a, w, t0 == 0), cols = int64_t(it.n) * a.per;
            CHECK(cols <= a.split_cols && at + cols <= static_cast<int64_t>(used.size()));
            for (int64_t c = at; c < at + cols; ++c) {
                CHECK(used[c] == -1);
                used[c] = w;
            }
            if (it.first < 0) it.first = w;
            ++it.pieces;
            ++kept;
            prefix_pieces += awq::kv_is_prefix(a, it.b);
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
static hipError_t seen(const KvAttend &a, bool split, bool wide, bool merge) {
    ++launched;
    CHECK(a.view && (a.view->sinks > 0) != (a.view->prefix.len != nullptr));
    ranges.clear();
    const int64_t H = a.c.heads, D = a.c.dim, heads = int64_t(a.s.T) * a.q_heads;
    const bool prefix = a.view->prefix.len != nullptr;
    if (merge) {
        CHECK(split);
        own(a.items, (a.s.B + (prefix ? 1 : 0)) * H * 8);
        own(a.part_ml, int64_t(a.workers) * 2 * a.split_cols * 8);
        own(a.part, int64_t(a.workers) * 2 * a.split_cols * D * 4);
    }
    if (a.wide_items) {
        const int64_t on_line = a.units - a.view->prefix.items_from;
        CHECK(wide && a.line && on_line > 0 && on_line * H < kKvLineUnits);
        lines_apart += a.view->prefix.items_from > 0;
        const int64_t n = int64_t(a.wide_workers) * 2 * kv_wide_cols(a.c.dim);
        own(a.wide_items, on_line * H * 8);
        own(a.wide_ml, n * 8);
        own(a.wide_part, n * D * 4);
    }
    if (prefix) {
        const KvPrefix &p = a.view->prefix;
        own(p.own, heads * D * 4);
        own(p.own_ml, heads * 8);
        own(p.common, heads * D * 4);
        own(p.common_ml, heads * 8);
        const int64_t all = int64_t(a.s.T) * a.per, cols = kv_wide_cols(a.c.dim);
        CHECK(a.units - p.own_units == (all > kv_split_cols(a.c.dim) ? (all + cols - 1) / cols : 0));
        CHECK(!a.window && (all > kv_split_cols(a.c.dim) || (split && all <= a.split_cols)));
        KvAttendPrefix v;
        static_cast<KvAttend &>(v) = a;
        v.p = p;
        if (split) walk(v, merge);
    } else {
        KvAttendSinks v;
        static_cast<KvAttend &>(v) = a;
        v.sinks = a.view->sinks;
        if (split) walk(v, merge);
    }
    return hipSuccess;
}
hipError_t launch_kv_attend_64(const KvAttend &a, int, bool s, bool w, bool m, hipStream_t) { return seen(a, s, w, m); }
hipError_t launch_kv_attend_128(const KvAttend &a, int, bool s, bool w, bool m, hipStream_t) { return seen(a, s, w, m); }
hipError_t launch_kv_attend_256(const KvAttend &a, int, bool s, bool w, bool m, hipStream_t) { return seen(a, s, w, m); }
hipError_t launch_kv_append(const KvCache &, const KvBatch &, const void *, const void *, int, int64_t, int64_t, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_kv_read(const KvCache &, const KvBatch &, void *, void *, int, int64_t, int64_t, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_kv_append_rotated(const KvCache &c, const KvBatch &s, const KvTurn &t, const void *, const void *, const void *,
                                    void *, int, int q_heads, int64_t, int64_t, int64_t, int64_t, hipStream_t) {
    ++launched;
    CHECK(s.T > 0 && q_heads > 0 && t.rot >= 0 && t.rot <= c.dim && t.rot % 16 == 0);
    CHECK((t.rot == 0 || t.positions > 0) && ((!t.q_weight && !t.k_weight) || t.eps > 0));
    return hipSuccess;
}
hipError_t launch_kv_tables(const KvTables &a, hipStream_t) {
    ++launched;
    CHECK(a.B > 0 && a.max_pages > 0 && (int64_t(a.max_pages) << a.page_shift) <= (int64_t(1) << 30) && a.T >= 0 && a.n_free >= 0);
    return hipSuccess;
}
}  // namespace awq

static void attention(std::mt19937 &rng, int round) {
    auto pick = [&](std::initializer_list<int> v) { return *(v.begin() + rng() % v.size()); };
    awq_kv_cache c{};
    c.pages = workspace, c.n_pages = 1 << 20, c.dim = pick({64, 128, 256}), c.group = pick({32, 64}), c.page = pick({16, 64, 256});
    c.heads = pick({1, 2, 5, 8});
    c.page_stride = static_cast<int64_t>(awq_kv_page_size(c.page, c.heads, c.dim, c.group));
    const int batch = pick({1, 2, 3, 17, 63, 64, 65, 130}), per = pick({1, 1, 2, 3, 4, 8, 16, 32, 71});
    const int span = pick({1, 6, 7, 40, 400}) * 64 / c.page + 1;
    const int max_rows = pick({1, 1, 1, 2, 3, 5, 8, 16, 0}), most = pick({1, 1, 2, 4, 16, 17, 64, 200});
    std::vector<int32_t> start(batch + 1), len(batch);
    for (int b = 0; b < batch; ++b) {
        const int n = rng() % 3 == 0 ? static_cast<int>(rng() % (most + 1)) : rng() % 8 == 0 ? 0 : 1;
        start[b + 1] = start[b] + n;
        len[b] = static_cast<int32_t>(rng() % 4 == 0 ? span * c.page : rng() % (span * c.page + 40));
    }
    awq_kv_batch s{};
    s.rows = start[batch] + rng() % 3, s.batch = batch, s.max_pages = span, s.kv_len = len.data(), s.block_table = len.data();
    s.row_start = start.data();
    if (round % 7 == 0) {
        s.row_start = nullptr;
        s.rows = int64_t(batch) * pick({1, 2, 5});
    } else if (round % 7 == 1) {   // nonsense, which the kernels bound
        for (auto &x : start) x = static_cast<int32_t>(rng());
        for (auto &x : len) x = static_cast<int32_t>(rng());
    }
    if (s.rows == 0) return;
    awq_kv_view view{};
    int32_t prefix_len = round % 5 == 0 ? static_cast<int32_t>(rng()) : static_cast<int32_t>(rng() % (span * c.page + 10));
    if (round % 2) {
        view.window = pick({1, 33, 200, 5000}), view.sinks = pick({1, 4, 32, 65, 1 << 30});
        if (round % 9 == 0) view.sinks = std::numeric_limits<int64_t>::max();
    } else {
        view.prefix_len = &prefix_len, view.prefix_table = len.data(), view.prefix_pages = pick({1, 2, 5, 30, 400});
    }
    const int64_t q_heads = per * c.heads;
    workspace_bytes = awq_kv_attention_workspace_size_ex(&c, &s, &view, q_heads, max_rows);
    const awq_status e = awq_kv_attention_ex(&c, &s, &view, workspace, AWQ_BF16, q_heads, q_heads * c.dim, max_rows, 1.0f, 1, workspace,
                                             q_heads * c.dim, nullptr, workspace, workspace_bytes, nullptr);
    if (e != AWQ_OK) std::printf("%s\n", awq_last_error());
    CHECK(e == AWQ_OK);
    if (workspace_bytes > 0)
        CHECK(awq_kv_attention_ex(&c, &s, &view, workspace, AWQ_BF16, q_heads, q_heads * c.dim, max_rows, 1.0f, 1, workspace,
                                  q_heads * c.dim, nullptr, workspace, workspace_bytes - 1, nullptr) == AWQ_ERR_WORKSPACE);
}

static void ends() {
    void *const P = workspace;
    const int64_t huge[] = {INT64_MAX, INT64_MIN, -1, 0, 1, 7, int64_t(1) << 20, int64_t(1) << 30, int64_t(1) << 31, int64_t(1) << 45};
    awq_kv_cache c{};
    c.pages = P, c.n_pages = 8, c.page_stride = 4 * 16 * 136, c.heads = 4, c.dim = 128, c.group = 128, c.page = 16;
    const int32_t *const I = static_cast<const int32_t *>(P);
    for (int64_t x : huge)
        for (int64_t y : huge) {
            awq_kv_batch s{};
            s.rows = x, s.batch = 1, s.max_pages = 4, s.kv_len = I, s.block_table = I;
            awq_kv_rotation r{};
            r.cos_sin = static_cast<const float *>(P), r.positions = y, r.rot = 64, r.eps = 1e-6;
            awq_kv_append_rotated(&c, &s, &r, P, P, P, AWQ_BF16, 8, 1024, 512, 512, P, 1024, nullptr);
            s.rows = 5, r.positions = 10;
            awq_kv_append_rotated(&c, &s, &r, P, P, P, AWQ_F32, x, y, 512, 512, P, y, nullptr);
            r.rot = static_cast<int>(x), r.interleaved = static_cast<int>(y);
            awq_kv_append_rotated(&c, &s, &r, P, P, P, AWQ_F16, 8, 1024, 512, 512, P, 1024, nullptr);
            r.rot = 0, r.interleaved = 0, r.q_weight = r.cos_sin;
            for (double eps : {0.0, -1.0, 1e-300, 1e300, std::nan(""), double(INFINITY)}) {
                r.eps = eps;
                const awq_status e = awq_kv_append_rotated(&c, &s, &r, P, P, P, AWQ_F16, 8, 1024, 512, 512, P, 1024, nullptr);
                CHECK(e == (eps > 0 && std::isfinite(eps) ? AWQ_OK : AWQ_ERR_ARG));
            }
            int32_t in[4], out[4];
            int64_t slot[1];
            const awq_kv_step step{out, out + 1, out + 2, out + 3, slot};
            awq_kv_tables(16, x, y, in, in + 1, in + 2, 5, in + 3, static_cast<int32_t *>(P), 7, &step, nullptr);
            awq_kv_tables(static_cast<int>(x), 3, 4, in, in + 1, in + 2, y, nullptr, static_cast<int32_t *>(P), 7, &step, nullptr);
            awq_kv_tables(256, 3, 4, in, in + 1, in + 2, x, in + 3, static_cast<int32_t *>(P), y, &step, nullptr);
        }
}

int main() {
    std::mt19937 rng(1);
    for (int round = 0; round < 12000; ++round) attention(rng, round);
    ends();
    CHECK(kept > 10000 && prefix_pieces > 1000 && sink_items > 1000 && launched > 12000 && lines_apart > 100);
    std::printf("%lld walks, %lld pieces in their places, %lld of a prefix, %lld items with sinks, %lld lines of a prefix alone\n", walks, kept, prefix_pieces, sink_items, lines_apart);
    return 0;
}
