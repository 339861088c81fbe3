// Internal declarations of the 4-bit key/value cache (k_kv*.hip, kv_attend.h, awq_kv*.hip).
//
// One block of bytes per (page, head), blocks of a page in head order, page
// size P tokens, D channels, groups of `group` channels, NG = D / group:
//   key codes    [P][D/2]           word kb*(D/32) + j of a token: channels 32j + 8kb + 0..7
//                                   in the nibble order 0,2,4,6,1,3,5,7 of k_pack.hip
//   value codes  [P/4][16][D/32][4] byte [t/4][m][b][t%4]: channel 32b + m (low nibble)
//                                   and 32b + 16 + m (high nibble) of token t
//   key pairs    [P][NG][2] fp16    (step, lowest value)
//   value pairs  [P][NG][2] fp16
//
// The codes lie as the matrix cores take them.  S^T = K·Q^T: lane (n, kb) of a
// 16x16x32 MFMA feeds 8 channels of key token n, so a lane's chunk kb of a
// token (D/32 words) is its operand for all D/32 MFMAs, one wide load.
// O^T = V^T·P^T: the lane that holds the scores of tokens 4kb..4kb+3 (the
// result rows of the first product) feeds the same tokens of value channel
// m, which are the bytes of its chunk [t/4][m]: scores go from the first
// product to the second without crossing lanes, and every wave load of codes
// is contiguous.
#pragma once

#include "awq_internal.h"

namespace awq {

struct KvCache {
    unsigned char *pages;
    int64_t page_stride;   // bytes between pages
    int64_t block;         // bytes of one (page, head)
    int n_pages, page_shift, heads, dim, group;
};

// The sequences of a call: sequence b's new rows are row_start[b] ..
// row_start[b+1] - 1 (b*even .. with row_start NULL), the last of its
// kv_len[b] positions.
struct KvBatch {
    const int32_t *row_start, *kv_len, *table;
    int B, max_pages, T, even;
};

constexpr float kKvMaxAbs = 32768.0f;   // larger values (and NaN) are stored as NaN

__host__ __device__ __forceinline__ int kv_clamp(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// First row and number of rows of sequence b, inside [0, T) whatever the table holds.
__host__ __device__ __forceinline__ void kv_rows(const KvBatch &s, int b, int &r0, int &n) {
    if (!s.row_start) {
        r0 = b * s.even;
        n = s.even;
        return;
    }
    r0 = kv_clamp(s.row_start[b], 0, s.T);
    n = kv_clamp(s.row_start[b + 1], r0, s.T) - r0;
}

// Tokens of sequence b, inside what its row of the page table holds.
__host__ __device__ __forceinline__ int kv_length(const KvBatch &s, int b, int page_shift) {
    return kv_clamp(s.kv_len[b], 0, s.max_pages << page_shift);
}

// Ragged rows in units of `size` (rows, or columns of `per` to a row): sequence
// b owns units first(b) .. first(b+1) - 1 with first(b) = start(b)*per / size +
// extra*b, which leaves room for every unit that its rows touch.  Finds the
// sequence of unit u.
__host__ __device__ __forceinline__ int kv_unit_first(const KvBatch &s, int b, int per, int size, int extra) {
    return static_cast<int>(static_cast<int64_t>(kv_clamp(s.row_start[b], 0, s.T)) * per / size) + extra * b;
}
__host__ __device__ __forceinline__ int kv_unit_sequence(const KvBatch &s, int u, int per, int size, int extra) {
    int lo = 0, hi = s.B;   // the last b in [0, B) with first(b) <= u
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (kv_unit_first(s, mid, per, size, extra) <= u)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// kv_unit_sequence (1, SIZE, EXTRA) of a unit that is one for the wave, all of whose lanes call:
// 64 sequences to a load, so that up to 64 cost one load's latency and not the six of a
// search by halves (reading 4 sequences of up to 16384: 22.8 -> 21.5 us).  SIZE, EXTRA: of the
// units (1 and 0: single rows).
template <int SIZE = 4, int EXTRA = 2>
__device__ __forceinline__ int kv_wave_sequence(const KvBatch &s, int unit, int lane) {
    int lo = 0, n = s.B;
    while (n > 1) {
        const int step = (n + 63) >> 6, at = lane * step;
        const int begun = __popcll(__ballot(at < n && kv_unit_first(s, lo + (at < n ? at : 0), 1, SIZE, EXTRA) <= unit));
        const int from = begun > 0 ? (begun - 1) * step : 0;
        lo += from;
        n = n - from < step ? n - from : step;
        if (begun == 0) break;   // (the first rows belong to no sequence)
    }
    return lo;
}

// A prefix that all sequences share is one more sequence, number B, behind the others: all rows
// of the call over the prefix's pages.  The others begin at its end.  All sums then go to
// memory, and one launch joins a row's own with the prefix's.
struct KvPrefix {
    const int32_t *len, *table;       // [1], [max_pages]
    int max_pages, own_units;         // own_units: of the wide path, before the prefix's
    int items_from;                   // units without a place in wide_items: 0, or own_units where the prefix's
                                      // form a line of their own in a launch of their own
    float *own, *own_ml;              // [T][q_heads][dim] and [..][2]: sums of items that were not cut
    float *common, *common_ml;        // the same of the prefix
};
struct KvView {
    int sinks;                        // first positions that stay visible under the window
    KvPrefix prefix;                  // len NULL: none
};

struct KvAttend {
    KvCache c;
    KvBatch s;
    const void *Q;
    void *O;
    float *lse;
    int64_t q_stride, o_stride;   // elements between rows
    int q_heads, per;             // query heads, and query heads per key head
    float scale_log2;             // scale * log2(e)
    int causal, window;
    int split_cols;               // sequences with at most this many columns take the split path; a
                                  // piece's place in the workspace holds as many
    // split path
    int tiles_col;                // column tiles of 16 per item: 1, 2 or 4
    int workers;
    int snap;                     // tiles: pieces this short are not cut off
    int2 *items;                  // [kv_count*heads]: first worker and number of pieces (0: written already)
    float *part, *part_ml;        // [workers][2][split_cols][dim] and [..][2]
    // wide path
    int units, line, wide_workers;
    int2 *wide_items;             // [units*heads], as items; NULL where no unit is cut
    float *wide_part, *wide_ml;   // [wide_workers][2][kv_wide_cols][dim] and [..][2]
    const KvView *view;           // (host memory) NULL: none
};

// The arguments of the kernels with sinks, and with a shared prefix.  Kernels and their functions
// take any of the three types, A; what only one of them has is a constant for the others, so
// that calls without it pay nothing for it.  (One kernel for all cost calls without either 3% on
// long caches, 5% at dim 256 and 23%, 4 us, on items of few tiles; fields set to constants in a
// copy of the arguments, which is then held in registers, half of that.)
struct KvAttendSinks : KvAttend {
    int sinks;
};
struct KvAttendPrefix : KvAttend {
    KvPrefix p;
};
__host__ __device__ __forceinline__ int kv_sinks(const KvAttend &) { return 0; }
__host__ __device__ __forceinline__ int kv_sinks(const KvAttendSinks &a) { return a.sinks; }
// Sequences, the prefix among them.
__host__ __device__ __forceinline__ int kv_count(const KvAttend &a) { return a.s.B; }
__host__ __device__ __forceinline__ int kv_count(const KvAttendPrefix &a) { return a.s.B + 1; }
__host__ __device__ __forceinline__ bool kv_is_prefix(const KvAttend &, int) { return false; }
__host__ __device__ __forceinline__ bool kv_is_prefix(const KvAttendPrefix &a, int b) { return b == a.s.B; }
// Positions of the prefix.
__host__ __device__ __forceinline__ int kv_common(const KvAttend &) { return 0; }
__host__ __device__ __forceinline__ int kv_common(const KvAttendPrefix &a) {
    return kv_clamp(*a.p.len, 0, a.p.max_pages << a.c.page_shift);
}
// Rows, length and pages of sequence b.
__host__ __device__ __forceinline__ void kv_sequence(const KvAttend &a, int b, int, int &r0, int &n, int &len) {
    kv_rows(a.s, b, r0, n);
    len = kv_length(a.s, b, a.c.page_shift);
}
__host__ __device__ __forceinline__ void kv_sequence(const KvAttendPrefix &a, int b, int common, int &r0, int &n, int &len) {
    if (b == a.s.B) {
        r0 = 0, n = a.s.T, len = common;
        return;
    }
    kv_sequence(static_cast<const KvAttend &>(a), b, common, r0, n, len);
}
__host__ __device__ __forceinline__ const int32_t *kv_table(const KvAttend &a, int b) {
    return a.s.table + static_cast<int64_t>(b) * a.s.max_pages;
}
__host__ __device__ __forceinline__ const int32_t *kv_table(const KvAttendPrefix &a, int b) {
    return b == a.s.B ? a.p.table : kv_table(static_cast<const KvAttend &>(a), b);
}

// A sequence's columns are its query rows x the query heads of one key head.
// Most columns of the split path (4 column tiles of 16, or 2 at dim 256, where the
// output of 4 does not fit the registers).  16 sequences of 4096 tokens, 8 key heads:
// at dim 128 64 columns take 76 us on it and 97 on the wide path, 32 columns 46 and
// 100; at dim 64 64 columns 49 and 76; at dim 256 (4 heads) 32 columns 59 and 90.
constexpr int kv_split_cols(int dim) { return dim > 128 ? 32 : 64; }
// Columns of one workgroup of the wide path, 32 to a wave: 8 waves, or 4 where
// the output alone takes 128 registers.
constexpr int kv_wide_cols(int dim) { return dim > 128 ? 128 : 256; }
constexpr int kv_wide_tile(int dim) { return 8192 / dim; }   // tokens
constexpr int kKvCus = 256;          // a workgroup of the wide path fills a CU
// With fewer (unit, head)s than this they may form a line; from 2 to a CU on, the
// longest first load the GPU evenly without its pieces.  (128 rows over 32768 tokens:
// 109 us on the line, 1198 us without; 5 ragged chunks at dim 256: 256 and 395 us; a
// prompt of 4096, 512 units: 243 and 184 us.)
constexpr int kKvLineUnits = 2 * kKvCus;
// What a piece of a unit costs besides its tiles, in tiles (13 to 15 us of a chain of waits; a tile
// takes 3.3 us at dim 64, 2.5 at 128 and 2.0 at 256), and what the join of cut units costs (its
// launch and the sums' way through memory).  Whole units are handed out where that is no slower
// than the line by these: 5 ragged chunks over 6007 tokens at dim 256 take 258 us, and 304 with costs
// of 3 and the line up to 6/5 of its time; the same under a window 96 and 106; 6 random prompts of up to
// 700 rows over 6000 at dim 64, 128 and 256 200, 257 and 820 us both ways.
constexpr int kv_wide_cost(int dim) { return dim > 128 ? 7 : dim > 64 ? 5 : 4; }
constexpr int kKvWideMerge = 3;
// Least share of a workgroup, in tiles (4: 16 chunks of 64 rows over 512 tokens 43 -> 50 us; 8: one of
// them over 1024 38 -> 58).
constexpr int kKvWideMinShare = 6;
constexpr int kKvWideSnap = 1;       // tiles: pieces this short are not cut off (3: prompts 2% slower)
constexpr int kKvWideJoin = 2048;    // workgroups of the join of cut units, about (kv_attend.h)
constexpr int kKvTile = 32;        // tokens of one step
constexpr int kKvItemCost = 2;     // what an item costs besides its tiles, in tiles
// Least share of a worker, in tiles: a worker's part costs as much as about 2 tiles,
// but latency is what the small calls pay (one sequence of 65 tokens, 8 tiles instead
// of 4: 11.8 us instead of 7.4; 64 of up to 8192: 31.9 instead of 30.0).
constexpr int kKvMinShare = 4;
constexpr int kKvSnap = 1;         // tiles: pieces this short are not cut off (2 * snap < least share)
// Where no item can be longer (in tiles), none is cut: that saves the join, a launch of
// 3 to 4 us (one sequence, 8 heads of 128: 4 tiles 12.4 us cut and 9.0 whole, 8 tiles 12.6
// and 13.1, 12 tiles 12.5 and 17.5; heads of 256: 16.7 and 13.0, 16.5 and 20.6).
constexpr int kKvWhole = 6;
// Up to so many columns (of all items) have their pieces joined 32 channels to a
// workgroup: few columns have many pieces each, which more workgroups read sooner (64
// columns, dim 128, 131072 tokens: 52.5 -> 48.0 us in all; dim 256, 65536: 42.1 -> 34.0);
// many are quicker with fewer workgroups (512 columns: 43.6 us and 44.9; 4096: 29.5 and 36.8).
constexpr int kKvMergeFew = 256;
// The join of a call with a prefix: up to kKvMergeFew columns (row and query head) are spread as above,
// up to kKvJoinFew take a wave each, whose 256/dim groups share a column's pieces, and more take dim/4
// threads each.  What decides is the pieces of a column: n columns have up to 65536/n of the prefix's
// (32768/n at dim 256, where the two forms are one), as many as share the line's 256 workgroups, but
// behind a short prefix fewer, which the host does not know.  Wave and dim/4 threads, us:
//   columns of      3 pieces             8                    16
//   dim 64   2048   4.6  4.6             4.7  5.5             5.5  7.2
//            4096   4.8  4.6             5.8  5.8             7.1  7.9
//            8192   7.3  4.6             8.4  6.6
//   dim 128  2048   4.6  4.6             4.9  4.9             6.2  6.7
//            4096   5.1  4.5             6.4  5.2             9.0  8.5 (64 rows over 16384 positions: 10.4 12.6)
//            8192   7.7  5.0             9.4  8.1
// So the wave is the quicker one for many pieces, which there are up to about the bound, and costs up to 1.2 us
// at it behind short prefixes.
constexpr int64_t kKvJoinFew = 4096;
// Waves of the split path that a SIMD holds at once, by the registers of a wave's
// output (dim x 16*NT columns) and what comes with it: as many as do without spills, since
// they hide each other's latency.  us with 1 / 2 / 3 / 4, at group 32 (the largest group has the
// same fastest): dim 64 (8 heads), NT 1 (64 sequences of 4096) 108 / 69 / 60 / 53, NT 2
// (16 of 4096) 47 / 36 / 31 / 45, NT 4 (16 of 4096) 61 / 47 / 87 / 215; dim 128 (8 heads), NT 1 (131072
// tokens) 72 / 52 / 47 / 56, NT 2 (16 of 4096) 57 / 46 / 90 / 196, NT 4 (24 of 4096) 118 / 289 / 602 / 744;
// dim 256 (4 heads), NT 1 (48 of 4096) 98 / 70 / 203 / 294, NT 2 (16 of 4096) 59 / 144 / 236 / 289.
constexpr int kv_split_waves(int dim, int nt) {
    return nt * dim <= 64 ? 4 : nt * dim <= 128 ? 3 : nt * dim <= 256 ? 2 : 1;
}

// First position behind the sinks that any of a sequence's rows sees: what lies before it is
// treated as what lies behind its length, whatever its slots hold.  common: positions of the
// prefix that are not the sequence's own.
__host__ __device__ __forceinline__ int kv_lowest(const KvAttend &a, int len, int n, int) {
    if (!a.window) return 0;
    const int low = len - n - a.window + 1;
    return low > 0 ? low : 0;
}
__host__ __device__ __forceinline__ int kv_lowest(const KvAttendPrefix &, int len, int, int common) {
    return common < len ? common : len;
}
// The same of the row at position len - n + i; not bounded.
__host__ __device__ __forceinline__ int kv_low(const KvAttend &a, int len, int n, int i, int) {
    return a.window ? len - n + i - a.window + 1 : 0;
}
__host__ __device__ __forceinline__ int kv_low(const KvAttendPrefix &a, int len, int n, int, int common) {
    return kv_lowest(a, len, n, common);
}

// The split path's line (kv_attend.h).
template <typename A>
__host__ __device__ __forceinline__ int kv_first_token(const A &a, int len, int n, int common) {
    return kv_lowest(a, len, n, common) & ~(kKvTile - 1);
}
// Whole tiles of `tile` tokens before `first` (a multiple of it) that hold sinks.
template <typename A>
__host__ __device__ __forceinline__ int kv_sink_tiles(const A &a, int first, int tile) {
    if (kv_sinks(a) == 0) return 0;
    const int n = (kv_sinks(a) + tile - 1) / tile;
    return n < first / tile ? n : first / tile;
}
// Tiles of an item of sequence b, the sinks' first; 0: not on the split path.
template <typename A>
__host__ __device__ __forceinline__ int kv_item_tiles(const A &a, int b, int &r0, int &n, int &len, int common = 0) {
    kv_sequence(a, b, common, r0, n, len);
    if (n == 0 || static_cast<int64_t>(n) * a.per > a.split_cols) return 0;
    const int first = kv_first_token(a, len, n, kv_is_prefix(a, b) ? 0 : common), t = (len - first + kKvTile - 1) / kKvTile;
    return kv_sink_tiles(a, first, kKvTile) + (t > 0 ? t : 1);   // an empty item is visited, too: its output is zero
}
// Workers that share a line of this length, and where worker w's share begins (w = workers: the line's end).
__host__ __device__ __forceinline__ int kv_workers(const KvAttend &a, int total) {
    const int most = total / kKvMinShare > 1 ? total / kKvMinShare : 1;
    return a.workers < most ? a.workers : most;
}
// (w * total / workers, rounded down; with at most 2^15 workers nothing passes 32 bits, where a
// division takes a tenth of the instructions of one of 64.)
__host__ __device__ __forceinline__ int kv_share(int w, int total, int workers) {
    const uint32_t each = static_cast<uint32_t>(total) / static_cast<uint32_t>(workers), rest = total - each * workers;
    return static_cast<int>(w * each + w * rest / static_cast<uint32_t>(workers));
}
// The tile at which a boundary at x cuts an item that begins at `begin` (0 or tiles: not inside).
__host__ __device__ __forceinline__ int kv_cut(const KvAttend &a, int begin, int tiles, int x) {
    const int t = x - begin - kKvItemCost;
    if (t <= a.snap) return 0;
    return tiles - t <= a.snap ? tiles : t;
}
// First column of a piece in the workspace: of a worker's two, the one that begins its item goes second.
__host__ __device__ __forceinline__ int64_t kv_piece(const KvAttend &a, int worker, bool begins) {
    return (static_cast<int64_t>(worker) * 2 + (begins ? 1 : 0)) * a.split_cols;
}

// The wide path's units and line (kv_attend.h).
// Unit u: a sequence's columns col0 .. (kv_wide_cols(D) of them at most), and the
// tiles t0 .. t1-1 that some of them see (one at least, so that every unit is visited).
// Tiles before sink_tiles (with sinks, t0 is 0) lie at t, the others `skip` tiles further on.
struct KvUnit {
    int b, r0, n, len, col0, t0, t1, sink_tiles, skip;
};
// Units of the sequences themselves; those of a prefix come behind them.
__host__ __device__ __forceinline__ int kv_own_units(const KvAttend &a) { return a.units; }
__host__ __device__ __forceinline__ int kv_own_units(const KvAttendPrefix &a) { return a.p.own_units; }
template <int D, typename A>
__host__ __device__ __forceinline__ bool kv_unit(const A &a, int u, int common, KvUnit &x) {
    constexpr int kCols = kv_wide_cols(D), TT = kv_wide_tile(D);
    int k;
    if (u >= kv_own_units(a)) {
        x.b = a.s.B;
        k = u - kv_own_units(a);
    } else if (a.s.row_start) {
        x.b = kv_unit_sequence(a.s, u, a.per, kCols, 1);
        k = u - kv_unit_first(a.s, x.b, a.per, kCols, 1);
    } else {
        const int each = kv_own_units(a) / a.s.B;
        x.b = u / each;
        k = u - x.b * each;
    }
    if (x.b >= kv_count(a)) return false;   // (not in any launch)
    kv_sequence(a, x.b, common, x.r0, x.n, x.len);
    const bool prefix = kv_is_prefix(a, x.b);
    const int64_t cols = static_cast<int64_t>(x.n) * a.per;
    if (cols <= a.split_cols || k < 0 || static_cast<int64_t>(k) * kCols >= cols) return false;
    x.col0 = k * kCols;
    const int p0 = x.len - x.n, last = static_cast<int>(cols) - 1;
    const int end = x.col0 + kCols - 1 < last ? x.col0 + kCols - 1 : last;
    const int lo = kv_low(a, x.len, x.n, x.col0 / a.per, prefix ? 0 : common);
    const int hi = a.causal && !prefix ? p0 + end / a.per + 1 : x.len;
    x.t0 = lo > 0 ? lo / TT : 0;
    x.t1 = hi > 0 ? (hi + TT - 1) / TT : 0;
    if (x.t1 <= x.t0) x.t1 = x.t0 + 1;
    x.sink_tiles = kv_sink_tiles(a, x.t0 * TT, TT);
    x.skip = 0;
    if (x.sink_tiles > 0) {
        x.skip = x.t0 - x.sink_tiles;
        x.t1 -= x.skip;
        x.t0 = 0;
    }
    return true;
}
// Workgroups that share a line of this length.
__host__ __device__ __forceinline__ int kv_wide_workers(const KvAttend &a, int total) {
    const int most = total / kKvWideMinShare > 1 ? total / kKvWideMinShare : 1;
    return a.wide_workers < most ? a.wide_workers : most;
}
// The tile at which a boundary `at` behind an item's begin cuts it (0 or tiles: not inside).
template <int D>
__host__ __device__ __forceinline__ int kv_wide_cut(int at, int tiles) {
    const int t = at - kv_wide_cost(D);
    if (t <= kKvWideSnap) return 0;
    return tiles - t <= kKvWideSnap ? tiles : t;
}
// Whether pieces of a line are done sooner than whole units, of which some workgroup's take `time`.
template <int D>
__host__ __device__ __forceinline__ bool kv_wide_sooner(const KvAttend &a, int time, int line) {
    return (time - kv_wide_cost(D) - kKvWideMerge) * static_cast<int64_t>(kv_wide_workers(a, line)) > line;
}

// The join of a call with a prefix (kv_attend.h).
// Where the sums of one column lie: `count` pieces, the first (which begins the item) at `first`, the
// others `step` further on each, of places of D channels; or one place in `part` (count 1, first 0).
struct KvParts {
    const float *ml, *part;
    int64_t first, next;   // the first piece's place, and the second's
    int64_t step;          // from the second on
    int count;
};
template <int D>
__host__ __device__ __forceinline__ KvParts kv_parts(const KvAttendPrefix &a, int b, int r0, int n, int row, int qh, bool prefix) {
    const int head = qh / a.per, col = (row - r0) * a.per + (qh - head * a.per);
    const int64_t at = static_cast<int64_t>(row) * a.q_heads + qh;
    KvParts p = {prefix ? a.p.common_ml : a.p.own_ml, prefix ? a.p.common : a.p.own, at, at, 0, 1};
    if (static_cast<int64_t>(n) * a.per <= a.split_cols) {
        const int2 it = a.items ? a.items[b * a.c.heads + head] : make_int2(0, 0);
        if (it.y > 0 && it.x >= 0 && it.x < a.workers) {
            p.ml = a.part_ml, p.part = a.part;
            p.first = kv_piece(a, it.x, true) + col;
            p.next = kv_piece(a, it.x + 1, false) + col;
            p.step = 2 * a.split_cols;
            p.count = it.y < a.workers - it.x ? it.y : a.workers - it.x;   // (inside, should tables change under the call)
        }
        return p;
    }
    constexpr int kCols = kv_wide_cols(D);
    int unit;
    if (prefix)
        unit = a.p.own_units;
    else if (a.s.row_start)
        unit = kv_unit_first(a.s, b, a.per, kCols, 1);
    else
        unit = b * (a.p.own_units / a.s.B);
    unit += col / kCols;
    const int record = unit - a.p.items_from;
    const int2 it = a.wide_items && record >= 0 && unit < a.units ? a.wide_items[static_cast<int64_t>(record) * a.c.heads + head] : make_int2(0, 0);
    if (it.y > 0 && it.x >= 0 && it.x < a.wide_workers) {
        p.ml = a.wide_ml, p.part = a.wide_part;
        p.first = (2 * static_cast<int64_t>(it.x) + 1) * kCols + col % kCols;
        p.next = 2 * (static_cast<int64_t>(it.x) + 1) * kCols + col % kCols;
        p.step = 2 * kCols;
        p.count = it.y < a.wide_workers - it.x ? it.y : a.wide_workers - it.x;
    }
    return p;
}

// Norms and rotation of kv_append_rotated (k_kv_rotate.hip).
struct KvTurn {
    const float *cos_sin;              // [positions][2][rot/2]
    int positions, rot, neighbours;
    const float *q_weight, *k_weight;  // [dim], NULL: no norm
    double eps;
    bool keys_first;                   // queries are written where keys or values lie: only when those have been read
};

// A step's tables (k_kv_tables.hip).
struct KvTables {
    const int32_t *kv_len, *count, *free_pages, *taken;
    int64_t n_free, T;
    int32_t *table, *new_len, *row_start, *new_taken, *position;
    int64_t *slot, n_pages;            // pages from n_pages on have no slots
    int B, max_pages, page_shift;
};

hipError_t launch_kv_append_rotated(const KvCache &c, const KvBatch &s, const KvTurn &t, const void *Q, const void *K,
                                    const void *V, void *Qo, int type, int q_heads, int64_t q_stride, int64_t k_stride,
                                    int64_t v_stride, int64_t o_stride, hipStream_t st);
hipError_t launch_kv_tables(const KvTables &a, hipStream_t st);
hipError_t launch_kv_append(const KvCache &c, const KvBatch &s, const void *K, const void *V, int type,
                            int64_t k_stride, int64_t v_stride, hipStream_t st);
hipError_t launch_kv_read(const KvCache &c, const KvBatch &s, void *K, void *V, int type, int64_t k_stride,
                          int64_t v_stride, hipStream_t st);
// run_split, run_wide, merge: the launches that the call needs (awq_kv.hip)
hipError_t launch_kv_attend_64(const KvAttend &a, int type, bool run_split, bool run_wide, bool merge, hipStream_t st);
hipError_t launch_kv_attend_128(const KvAttend &a, int type, bool run_split, bool run_wide, bool merge, hipStream_t st);
hipError_t launch_kv_attend_256(const KvAttend &a, int type, bool run_split, bool run_wide, bool merge, hipStream_t st);

}  // namespace awq
