// Internal declarations of the 4-bit key/value cache (k_kv.hip, kv_attend.h, awq_kv.hip).
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
__device__ __forceinline__ int kv_unit_first(const KvBatch &s, int b, int per, int size, int extra) {
    return static_cast<int>(static_cast<int64_t>(kv_clamp(s.row_start[b], 0, s.T)) * per / size) + extra * b;
}
__device__ __forceinline__ int kv_unit_sequence(const KvBatch &s, int u, int per, int size, int extra) {
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
    int2 *items;                  // [B*heads]: first worker and number of pieces (0: written already)
    float *part, *part_ml;        // [workers][2][split_cols][dim] and [..][2]
    // wide path
    int units, line, wide_workers;
    int2 *wide_items;             // [units*heads], as items; NULL where no unit is cut
    float *wide_part, *wide_ml;   // [wide_workers][2][kv_wide_cols][dim] and [..][2]
};

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
// 103 us on the line, 1044 us without; 5 ragged chunks at dim 256: 295 and 383 us; a
// prompt of 4096, 512 units: 243 and 199 us.)
constexpr int kKvLineUnits = 2 * kKvCus;
constexpr int kKvWideCost = 3;       // what a unit costs besides its tiles, in tiles
constexpr int kKvWideMinShare = 6;   // least share of a workgroup, in tiles (12: within 1%)
constexpr int kKvWideSnap = 1;       // tiles: pieces this short are not cut off
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

// First position that any of a sequence's rows sees: what lies before it is treated as
// what lies behind its length, whatever its slots hold.
__host__ __device__ __forceinline__ int kv_lowest(const KvAttend &a, int len, int n) {
    if (!a.window) return 0;
    const int low = len - n - a.window + 1;
    return low > 0 ? low : 0;
}

// The split path's line (kv_attend.h).
__host__ __device__ __forceinline__ int kv_first_token(const KvAttend &a, int len, int n) {
    return kv_lowest(a, len, n) & ~(kKvTile - 1);
}
// Tiles of an item of sequence b; 0: not on the split path.
__host__ __device__ __forceinline__ int kv_item_tiles(const KvAttend &a, int b, int &r0, int &n, int &len) {
    kv_rows(a.s, b, r0, n);
    len = kv_length(a.s, b, a.c.page_shift);
    if (n == 0 || static_cast<int64_t>(n) * a.per > a.split_cols) return 0;
    const int t = (len - kv_first_token(a, len, n) + kKvTile - 1) / kKvTile;
    return t > 0 ? t : 1;   // an empty item is visited, too: its output is zero
}
// Workers that share a line of this length, and where worker w's share begins (w = workers: the line's end).
__host__ __device__ __forceinline__ int kv_workers(const KvAttend &a, int total) {
    const int most = total / kKvMinShare > 1 ? total / kKvMinShare : 1;
    return a.workers < most ? a.workers : most;
}
__host__ __device__ __forceinline__ int kv_share(int w, int total, int workers) {
    return static_cast<int>(static_cast<int64_t>(w) * total / workers);
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

hipError_t launch_kv_append(const KvCache &c, const KvBatch &s, const void *K, const void *V, int type,
                            int64_t k_stride, int64_t v_stride, hipStream_t st);
hipError_t launch_kv_read(const KvCache &c, const KvBatch &s, void *K, void *V, int type, int64_t k_stride,
                          int64_t v_stride, hipStream_t st);
// run_split, run_wide, merge: the launches that the call needs (awq_kv.hip)
hipError_t launch_kv_attend_64(const KvAttend &a, int type, bool run_split, bool run_wide, bool merge, hipStream_t st);
hipError_t launch_kv_attend_128(const KvAttend &a, int type, bool run_split, bool run_wide, bool merge, hipStream_t st);
hipError_t launch_kv_attend_256(const KvAttend &a, int type, bool run_split, bool run_wide, bool merge, hipStream_t st);

}  // namespace awq
