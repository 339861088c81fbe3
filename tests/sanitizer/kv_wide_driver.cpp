// Walks calls of attention on the host as the kernels do, both paths, over the arguments that
// awq_kv_attention_ex hands to its launches: the wide path's units make up every sequence's columns, its
// line is handed out whole or cut into pieces that make up their units, each in a place of its own
// inside the workspace, and the records tell the joins where they lie; with a prefix, kv_parts leads
// from a row and query head to the places of its own sums and of the prefix's, in order.  No part of the workspace
// is larger than what its launch uses.  The launches are replaced by the walk; nothing reaches a device.
#include "awq.h"

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <tuple>
#include <type_traits>
#include <vector>

#include "kv_internal.h"

#define CHECK(x)                                                                        \
    do {                                                                                \
        if (!(x)) {                                                                     \
            std::printf("FAILED %s:%d: %s (round %d)\n", __FILE__, __LINE__, #x, now); \
            std::exit(1);                                                               \
        }                                                                               \
    } while (0)

static int now;
static size_t workspace_bytes;
static std::vector<unsigned char> room;
static bool sane;
static std::mt19937 rng(5);
static long long lines, lines_whole, lines_cut, alone, wide_pieces, units_seen, sink_units, apart_lines, columns_joined, split_joined, wide_joined;

struct Owner {   // of one place: whose sums it holds
    int b, head, col0, order;
    bool operator==(const Owner &o) const { return b == o.b && head == o.head && col0 == o.col0 && order == o.order; }
};
static std::map<int64_t, Owner> split_places, wide_places;         // by (worker, 0 or 1)
static std::set<std::tuple<int, int, int>> direct;                 // (sequence, head, first column) whose sums are whole

template <typename A>
static void walk_split(const A &a, bool merge) {
    struct Item { int b, head, tiles, begin, end, covered, first, count; };
    std::vector<Item> items;
    int total = 0;
    const int common = awq::kv_common(a), H = a.c.heads;
    for (int b = 0; b < awq::kv_count(a); ++b) {
        int r0, n, len;
        const int tiles = awq::kv_item_tiles(a, b, r0, n, len, common);
        for (int h = 0; h < H && tiles > 0; ++h) {
            items.push_back({b, h, tiles, total, total + tiles + awq::kKvItemCost, 0, -1, 0});
            total = items.back().end;
        }
    }
    if (total == 0) return;
    const int workers = awq::kv_workers(a, total);
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
            const bool whole = t0 == 0 && t1 == it.tiles;
            if (whole) {
                CHECK(direct.insert({it.b, it.head, 0}).second);
            } else {
                CHECK(merge);
                CHECK(split_places.insert({int64_t(w) * 2 + (t0 == 0), {it.b, it.head, 0, it.count}}).second);
                if (it.first < 0) it.first = w;
                ++it.count;
            }
            if (t0 == 0 && a.items) {
                const int last = static_cast<int>((static_cast<int64_t>(it.end - a.snap) * workers + total - 1) / total) - 1;
                a.items[it.b * H + it.head] = whole ? int2{0, 0} : int2{w, last - w + 1};
            }
        }
    }
    for (const Item &it : items) {
        CHECK(it.covered == it.tiles);
        if (a.items) CHECK(a.items[it.b * H + it.head].y == it.count && (it.count == 0 || a.items[it.b * H + it.head].x == it.first));
    }
}

// One launch of the wide kernel.
template <int D, typename A>
static void walk_wide(const A &a) {
    constexpr int kCols = awq::kv_wide_cols(D), TT = awq::kv_wide_tile(D);
    const int H = a.c.heads, common = awq::kv_common(a);
    const int grid = a.line && a.wide_workers > a.units * H ? a.wide_workers : a.units * H;
    std::vector<awq::KvUnit> units(a.units);
    std::vector<int> there(a.units), before(a.units + 1, 0);
    for (int u = 0; u < a.units; ++u) {
        awq::KvUnit &x = units[u];
        there[u] = awq::kv_unit<D>(a, u, common, x);
        before[u + 1] = before[u];
        if (!there[u]) continue;
        ++units_seen;
        sink_units += x.sink_tiles > 0;
        CHECK(x.b >= 0 && x.b < awq::kv_count(a) && x.r0 >= 0 && x.n > 0 && x.r0 + x.n <= a.s.T);
        CHECK(x.col0 >= 0 && x.col0 % kCols == 0 && int64_t(x.col0) < int64_t(x.n) * a.per);
        CHECK(x.t0 >= 0 && x.t1 > x.t0 && x.sink_tiles >= 0 && x.skip >= 0);
        // (tiles begin inside the length, or are the one that an empty unit visits)
        CHECK(int64_t(x.t1 - 1 + (x.sink_tiles > 0 ? x.skip : 0)) * TT <= x.len);
        CHECK(x.sink_tiles == 0 || (x.t0 == 0 && x.sink_tiles <= x.t1));
        before[u + 1] += x.t1 - x.t0 + awq::kv_wide_cost(D);
    }
    auto hold = [&](int u, int head) { CHECK(direct.insert({units[u].b, head, units[u].col0}).second); };
    if (!a.line) {
        ++alone;
        for (int u = 0; u < a.units; ++u)
            for (int h = 0; h < H && there[u]; ++h) hold(u, h);
        return;
    }
    ++lines;
    CHECK(a.units <= awq::kKvLineUnits && a.units * H < awq::kKvLineUnits);
    const int all = before[a.units], total = H * all;
    if (total == 0) return;
    const int some = static_cast<int>(std::count(there.begin(), there.end(), 1)), jobs = H * some;
    const int workers = awq::kv_wide_workers(a, total);
    CHECK(workers >= 1 && workers <= a.wide_workers && workers <= grid && jobs <= grid);
    bool pieces = awq::kv_wide_sooner<D>(a, static_cast<int>(uint32_t(all) / uint32_t(some)), H * all);
    std::vector<int> order(a.units, -1);
    if (!pieces) {
        for (int i = 0; i < a.units; ++i) {
            const int mine = before[i + 1] - before[i];
            int rank = 0;
            for (int j = 0; j < a.units; ++j) {
                const int length = before[j + 1] - before[j];
                rank += length > mine || (length == mine && j < i) ? 1 : 0;
            }
            CHECK(order[rank] == -1);
            order[rank] = i;
        }
        auto length = [&](int job) { return job >= jobs ? 0 : before[order[job / H] + 1] - before[order[job / H]]; };
        for (int i = 0; i < awq::kKvCus; ++i)
            pieces |= awq::kv_wide_sooner<D>(a, length(awq::kKvCus - 1 - i) + length(awq::kKvCus + i), H * all);
    }
    ++(pieces ? lines_cut : lines_whole);
    if (!pieces) {
        std::set<std::pair<int, int>> done;
        for (int block = 0; block < jobs; ++block) {
            const int u = order[block / H], head = block % H;
            CHECK(there[u] && done.insert({u, head}).second);
            hold(u, head);
            if (a.wide_items) a.wide_items[u * H + head] = int2{0, 0};
        }
        return;
    }
    std::vector<int> covered(size_t(a.units) * H, 0), first(covered.size(), -1), count(covered.size(), 0), told(covered.size(), 0);
    std::vector<int> seen(workers, 0);
    for (int block = 0; block < workers; ++block) {
        const int xcd = block & 7, rest = workers & 7, worker = xcd * (workers >> 3) + (xcd < rest ? xcd : rest) + (block >> 3);
        CHECK(worker >= 0 && worker < workers && !seen[worker]++);
    }
    for (int worker = 0; worker < workers; ++worker) {
        const int x0 = awq::kv_share(worker, total, workers), x1 = awq::kv_share(worker + 1, total, workers);
        for (int next = -1;;) {
            const int at = next < 0 ? x0 : next, head = awq::kv_clamp(at / all, 0, H - 1);
            int lo = 0, hi = a.units;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (head * all + before[mid] <= at) lo = mid; else hi = mid;
            }
            const int item = head * all + before[lo], length = before[lo + 1] - before[lo], tiles = length - awq::kv_wide_cost(D);
            CHECK(length > 0 && there[lo]);
            const int end = item + length;
            const int c0 = next < 0 ? awq::kv_wide_cut<D>(at - item, tiles) : 0;
            const int c1 = x1 >= end ? tiles : awq::kv_wide_cut<D>(x1 - item, tiles);
            const bool whole = c0 == 0 && c1 == tiles, more = end < x1;
            next = end;
            const int k = lo * H + head;
            if (c0 == 0 && c1 > 0) {
                const int last = static_cast<int>((static_cast<int64_t>(end - awq::kKvWideSnap) * workers + total - 1) / total) - 1;
                CHECK(!told[k]++);
                if (a.wide_items) a.wide_items[k] = whole ? int2{0, 0} : int2{worker, last - worker + 1};
            }
            if (c0 < c1) {
                CHECK(c0 == covered[k]);
                covered[k] = c1;
                if (whole) {
                    hold(lo, head);
                } else {
                    CHECK(a.wide_items);
                    CHECK(wide_places.insert({2 * int64_t(worker) + (c0 == 0), {units[lo].b, head, units[lo].col0, count[k]}}).second);
                    if (first[k] < 0) first[k] = worker;
                    ++count[k];
                    ++wide_pieces;
                }
            }
            if (!more) break;
        }
    }
    for (int u = 0; u < a.units; ++u)
        for (int h = 0; h < H && there[u]; ++h) {
            const int k = u * H + h;
            CHECK(covered[k] == units[u].t1 - units[u].t0 && told[k] == 1);
            if (a.wide_items) CHECK(a.wide_items[k].y == count[k] && (count[k] == 0 || a.wide_items[k].x == first[k]));
        }
}

// Every (sequence, head, unit's columns) of a call has its sums somewhere, once.
template <int D, typename A>
static void all_there(const A &a, bool own_wide) {
    constexpr int kCols = awq::kv_wide_cols(D);
    if (!sane) return;
    std::set<std::tuple<int, int, int>> held = direct;
    for (const auto *m : {&split_places, &wide_places})
        for (const auto &x : *m)
            if (x.second.order == 0) CHECK(held.insert({x.second.b, x.second.head, x.second.col0}).second);
    size_t want = 0;
    const int common = awq::kv_common(a);
    for (int b = 0; b < awq::kv_count(a); ++b) {
        int r0, n, len;
        awq::kv_sequence(a, b, common, r0, n, len);
        const int64_t cols = int64_t(n) * a.per;
        const bool wide = cols > a.split_cols;
        if (cols == 0 || (wide && !own_wide && !awq::kv_is_prefix(a, b))) continue;   // (more rows than said)
        for (int64_t c = 0; c < (wide ? cols : 1); c += kCols)
            for (int h = 0; h < a.c.heads; ++h, ++want) CHECK(held.count({b, h, static_cast<int>(c)}));
    }
    CHECK(want == held.size());
}

// What kv_parts says of single rows and query heads.
template <int D>
static void joined(const awq::KvAttendPrefix &a, bool own_wide) {
    constexpr int kCols = awq::kv_wide_cols(D);
    if (!sane) return;
    const int common = awq::kv_common(a);
    for (int i = 0; i < 60; ++i) {
        const int b = static_cast<int>(rng() % a.s.B), qh = static_cast<int>(rng() % a.q_heads);
        int r0, n, len;
        awq::kv_sequence(static_cast<const awq::KvAttend &>(a), b, common, r0, n, len);
        if (n == 0 || (int64_t(n) * a.per > a.split_cols && !own_wide)) continue;
        const int row = r0 + (i % 3 == 0 ? n - 1 : static_cast<int>(rng() % n)), head = qh / a.per;
        for (bool prefix : {false, true}) {
            const awq::KvParts p = prefix ? awq::kv_parts<D>(a, a.s.B, 0, a.s.T, row, qh, true) : awq::kv_parts<D>(a, b, r0, n, row, qh, false);
            const int seq = prefix ? a.s.B : b, rows = prefix ? a.s.T : n, col = (row - (prefix ? 0 : r0)) * a.per + qh % a.per;
            const bool wide = int64_t(rows) * a.per > a.split_cols;
            const int col0 = wide ? col / kCols * kCols : 0, cols = wide ? kCols : a.split_cols;
            ++columns_joined;
            if (direct.count({seq, head, col0})) {
                CHECK(p.part == (prefix ? a.p.common : a.p.own) && p.ml == (prefix ? a.p.common_ml : a.p.own_ml) && p.count == 1);
                CHECK(p.first == int64_t(row) * a.q_heads + qh);
                continue;
            }
            CHECK(p.part == (wide ? a.wide_part : a.part) && p.ml == (wide ? a.wide_ml : a.part_ml) && p.count > 1);
            ++(wide ? wide_joined : split_joined);
            for (int k = 0; k < p.count; ++k) {
                const int64_t at = k == 0 ? p.first : p.next + (k - 1) * p.step;
                CHECK(at % cols == col - col0);
                const auto &places = wide ? wide_places : split_places;
                const auto found = places.find(at / cols);
                CHECK(found != places.end() && found->second == (Owner{seq, head, col0, k}));
            }
            for (const auto &x : wide ? wide_places : split_places)
                if (x.second.b == seq && x.second.head == head && x.second.col0 == col0) CHECK(x.second.order < p.count);
        }
    }
}

template <int D>
static hipError_t seen(const awq::KvAttend &a, bool split, bool wide, bool merge) {
    split_places.clear(), wide_places.clear(), direct.clear();
    const int64_t H = a.c.heads, heads = int64_t(a.s.T) * a.q_heads;
    const bool prefix = a.view && a.view->prefix.len;
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    int64_t used = 0;
    if (merge) {
        const int64_t n = int64_t(a.workers) * 2 * a.split_cols;
        used += up((a.s.B + prefix) * H * 8) + up(n * 8) + up(n * D * 4);
    }
    if (a.wide_items) {
        const int64_t n = int64_t(a.wide_workers) * 2 * awq::kv_wide_cols(D);
        used += up((a.units - (prefix ? a.view->prefix.items_from : 0)) * H * 8) + up(n * 8) + up(n * D * 4);
    }
    if (prefix) used += 2 * (up(heads * 8) + up(heads * D * 4));
    CHECK(used == static_cast<int64_t>(workspace_bytes));
    if (prefix) {
        awq::KvAttendPrefix v;
        static_cast<awq::KvAttend &>(v) = a;
        v.p = a.view->prefix;
        if (split) walk_split(v, merge);
        if (wide) {
            awq::KvAttendPrefix w = v;
            if (v.p.items_from > 0) {
                ++apart_lines;
                w.units = v.p.own_units, w.line = 0, w.wide_items = nullptr;
                walk_wide<D>(w);
                w = v;
                w.units = v.units - v.p.own_units, w.p.own_units = 0;
            }
            walk_wide<D>(w);
        }
        all_there<D>(v, v.p.own_units > 0);
        joined<D>(v, v.p.own_units > 0);
    } else if (a.view) {
        awq::KvAttendSinks v;
        static_cast<awq::KvAttend &>(v) = a;
        v.sinks = a.view->sinks;
        if (split) walk_split(v, merge);
        if (wide) walk_wide<D>(v);
        all_there<D>(v, wide);
    } else {
        if (split) walk_split(a, merge);
        if (wide) walk_wide<D>(a);
        all_there<D>(a, wide);
    }
    return hipSuccess;
}

namespace awq {
hipError_t launch_kv_attend_64(const KvAttend &a, int, bool s, bool w, bool m, hipStream_t) { return seen<64>(a, s, w, m); }
hipError_t launch_kv_attend_128(const KvAttend &a, int, bool s, bool w, bool m, hipStream_t) { return seen<128>(a, s, w, m); }
hipError_t launch_kv_attend_256(const KvAttend &a, int, bool s, bool w, bool m, hipStream_t) { return seen<256>(a, s, w, m); }
hipError_t launch_kv_append(const KvCache &, const KvBatch &, const void *, const void *, int, int64_t, int64_t, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_kv_read(const KvCache &, const KvBatch &, void *, void *, int, int64_t, int64_t, hipStream_t) {
    return hipSuccess;
}
}  // namespace awq

static void call() {
    auto pick = [&](std::initializer_list<int> v) { return *(v.begin() + rng() % v.size()); };
    awq_kv_cache c{};
    c.pages = reinterpret_cast<void *>(uintptr_t(1) << 40), c.n_pages = 1 << 20, c.dim = pick({64, 128, 256}), c.group = 64, c.page = pick({16, 64});
    c.heads = pick({1, 2, 5, 8});
    c.page_stride = static_cast<int64_t>(awq_kv_page_size(c.page, c.heads, c.dim, c.group));
    const int batch = pick({1, 2, 3, 7, 17, 64, 100}), per = pick({1, 3, 4, 8, 16});
    const int span = pick({1, 8, 40, 150, 400}) * 64 / c.page, most = pick({1, 2, 40, 129, 300, 1000});
    std::vector<int32_t> start(batch + 1), len(batch);
    for (int b = 0; b < batch; ++b) {
        const int n = rng() % 3 == 0 ? static_cast<int>(rng() % (most + 1)) : rng() % 8 == 0 ? 0 : 1;
        start[b + 1] = start[b] + n;
        len[b] = static_cast<int32_t>(rng() % 4 == 0 ? span * c.page : rng() % (span * c.page + 40));
    }
    sane = true;
    awq_kv_batch s{};
    s.rows = start[batch] + rng() % 3, s.batch = batch, s.max_pages = span, s.kv_len = len.data(), s.block_table = len.data();
    s.row_start = start.data();
    if (now % 5 == 0) {
        s.row_start = nullptr;
        s.rows = int64_t(batch) * pick({1, 2, 5, 40, 300});
    } else if (now % 11 == 1) {   // nonsense, which the kernels bound
        sane = false;
        for (auto &x : start) x = static_cast<int32_t>(rng());
        for (auto &x : len) x = static_cast<int32_t>(rng());
    }
    if (s.rows == 0 || s.rows * per * c.heads > 400000) return;
    awq_kv_view view{};
    int32_t prefix_len = now % 13 == 0 ? static_cast<int32_t>(rng()) : static_cast<int32_t>(rng() % (span * c.page + 10));
    const int kind = now % 3;
    const int causal = kind == 1 ? 1 : pick({0, 1, 1});
    if (kind == 1)
        view.window = pick({1, 33, 200, 2000, 5000}), view.sinks = pick({0, 1, 4, 65, 129, 1 << 30});
    else if (kind == 2)
        view.prefix_len = &prefix_len, view.prefix_table = len.data(), view.prefix_pages = pick({1, 5, 30, 400});
    const int64_t q_heads = per * c.heads, max_rows = pick({0, 0, most, most, 1, 3});
    workspace_bytes = awq_kv_attention_workspace_size_ex(&c, &s, &view, q_heads, max_rows);
    if (room.size() < workspace_bytes + 16) room.resize(workspace_bytes + 16);
    unsigned char *const at = room.data() + (16 - reinterpret_cast<uintptr_t>(room.data()) % 16) % 16;
    void *const q = reinterpret_cast<void *>(uintptr_t(1) << 41);
    // (each row's real number is under max_rows, or its rows are left out)
    const awq_status e = awq_kv_attention_ex(&c, &s, &view, q, AWQ_BF16, q_heads, q_heads * c.dim, max_rows, 1.0f, causal, q, q_heads * c.dim,
                                             nullptr, at, workspace_bytes, nullptr);
    if (e != AWQ_OK) std::printf("%s\n", awq_last_error());
    CHECK(e == AWQ_OK);
}

int main() {
    for (now = 0; now < 6000; ++now) call();
    std::printf("%lld units (%lld with sinks), %lld without a line; %lld lines: %lld whole, %lld cut into %lld pieces, %lld of a prefix alone; "
                "%lld columns joined, %lld from pieces of the split path and %lld of the wide one\n",
                units_seen, sink_units, alone, lines, lines_whole, lines_cut, wide_pieces, apart_lines, columns_joined, split_joined, wide_joined);
    CHECK(alone > 300 && lines_whole > 300 && lines_cut > 300 && wide_pieces > 10000 && apart_lines > 30 && sink_units > 1000);
    CHECK(split_joined > 1000 && wide_joined > 1000);
    return 0;
}
