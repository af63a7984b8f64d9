// Which kernel form a grouped call takes: arithmetic on the call's sizes on the
// host, in functions of their own so that the tests can ask which form a size
// reaches.  The groups' ends are device data, so every rule goes by M and the
// number of groups; `full`, the most groups that can hold rows, stands for the
// groups that do.  `cus`: compute units of the device, 0 if unknown.
#pragma once

#include "mx_internal.h"

namespace mx {

inline int64_t full_groups(int64_t M, int groups) { return groups < M ? groups : M; }

// ------------------------------------------------------------ quantizers
constexpr int kQuantTile = 128;    // rows and columns of a quantize_kernel tile
constexpr int kEarlyIndex = 256;   // rows of an index that quantize_rows_kernel reads along with the ends

enum class QuantForm {
    kRows,     // quantize_rows_kernel: row-wise blob, units of 16 rows in order
    kSlices,   // quantize_slices_kernel: the same in slices of the groups
    kNarrow,   // quantize_narrow_kernel: both blobs, 128-row x 32-column tiles
    kTiles     // quantize_kernel: 128 x 128 tiles
};

// Workgroups of a quantize_rows_kernel launch.
inline int64_t quantize_rows_blocks(const QuantArgs &a) {
    return cdiv((a.M + 15 * full_groups(a.M, a.groups)) / 16 * cdiv(a.N_pad, 512), 4);
}

// The most 128-row tiles that M rows in a.groups groups can need.
inline int64_t quantize_row_tiles(const QuantArgs &a) {
    return (a.M + (kQuantTile - 1) * full_groups(a.M, a.groups)) / kQuantTile;
}

inline QuantForm quantize_form(const QuantArgs &a, bool dual, int cus) {
    if (!dual && !a.row.use_sr && !a.row.use_2d && !a.row.rht) {
        // More gathered rows than x has: some are read again.  In us, by units in
        // order / in slices, four inputs in turn: 512 rows of 1024 into 2 of 8 groups
        // 4.9 / 4.9, 777 of 1001 into 2 of 12 5.6 / 5.3, 2048 of 2048 into 4 of 64
        // 10.1 / 9.4, 16384 of 2048 into 2 of 16 29.5 / 27.6, 8192 of 2048 into 8 of 64
        // 47 / 39; into 1 of 64 (8192 of 4096, one input) 17.0 / 19.0.
        if (a.row_index && a.groups <= 64 && a.M > a.x_rows && a.M > kEarlyIndex && a.N_pad > 512 &&
            a.M < (int64_t(1) << 22))
            return QuantForm::kSlices;
        // (a grid holds fewer than 2^32 threads)
        if (quantize_rows_blocks(a) < int64_t(1) << 24) return QuantForm::kRows;
    }
    // In us, 128 x 128 tiles / narrow ones, full groups: 64 tiles 6.1 / 4.2 (SR 8.0
    // / 5.1), 256 tiles 6.3 / 7.1 (8.5 / 8.9), 512 tiles 8.4 / 10.5.  The count here
    // bounds ragged groups from above (a training step of 558 rows in 32 groups,
    // 1472 x 1216, 432 tiles by the bound, runs 105 / 98), so full groups of 256 to
    // 512 tiles, weights for instance, take the slower form.
    if (dual && !a.row.rht && !a.col.rht && quantize_row_tiles(a) * cdiv(a.N, kQuantTile) <= 2 * cus)
        return QuantForm::kNarrow;
    return QuantForm::kTiles;
}

// ------------------------------------------------------------ products
constexpr int kFewM = 64, kFewNB = 2, kFewN = 16 * kFewNB;   // tile of the few-rows form
constexpr int kStreamGroups = 512;                           // groups that the persistent form's table holds

enum class GemmForm {
    kFewRows,      // weights straight from memory to registers
    kTiles128,     // one 128x128 tile per workgroup
    kPersistent,   // one workgroup per CU, 256x256 tiles
    kTiles256      // one 256x256 tile per workgroup
};

// Most tiles of `tile` rows that M rows in `groups` groups and the rows
// behind the last group can need.
inline int64_t max_tiles(int64_t M, int groups, int tile) {
    return (M + (tile - 1) * (full_groups(M, groups) + 1)) / tile;
}

// Workgroups of the largest grid the entry points let through (a grid of
// 512-thread workgroups must stay below 2^32 threads).
constexpr int64_t kMaxBlocks = int64_t(1) << 22;

inline bool grouped_gemm_fits(int64_t M, int64_t N, int groups) {
    return max_tiles(M, groups, 128) * cdiv(N, 128) < kMaxBlocks;
}

inline bool grouped_wgrad_fits(int64_t N, int64_t K, int groups) {
    const int64_t tiles = cdiv(N, 128) * cdiv(K, 128);
    return tiles < kMaxBlocks && groups * tiles < kMaxBlocks;   // (the product alone can pass 64 bits)
}

// Whether the persistent form takes the product: bf16 output, a bias whose rows
// start at 16-byte boundaries, and 32-bit offsets into both blobs and a tile of
// C.
inline bool stream_fits(const GroupedGemmArgs &a, int64_t a_bytes, int64_t b_bytes) {
    constexpr int64_t kLimit = (int64_t(1) << 31) - 1;
    return a.out_dtype == MX_BF16 && a.groups <= kStreamGroups && a_bytes <= kLimit && b_bytes <= kLimit &&
           256 * a.ldc * 2 <= kLimit &&
           (!a.bias || (a.N % 8 == 0 && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0));
}

// Whether the persistent form takes its epilogue for any number of columns and
// row stride (ODD, cached stores) instead of the one for aligned rows
// (non-temporal ones).  Run in turn: 20510 rows of 809 columns, stride 816, K
// 1204 in 7 groups 42.7 us with its quantization, 46.9 with non-temporal stores;
// a training step of 16384 rows, 4096 x 2048 in 16 groups, takes 9% more with
// cached ones.
inline bool odd_rows(const GroupedGemmArgs &a, int64_t columns) { return columns % 8 != 0 || a.ldc % 64 != 0; }
inline bool wgrad_odd_rows(const GroupedGemmArgs &a) { return odd_rows(a, a.K) || a.group_stride % 64 != 0; }

// By the tiles that M rows would make with half a tile of padding in every
// group (the real spread is known on the device only).
// Measured on MI355X in us, few rows / 128x128 / persistent 256x256:
//   64 groups of 4, N 2048, K 4096    52 /  75 /  78
//   64 groups of 32                   68 /  77 /  79
//   64 groups of 64                   93 /  81 /  80
//   4 groups of 256, N 1200, K 1024  5.5 / 6.5 / 9.9
//   12 groups of 64                  5.2 / 6.0 / 9.7
//   12 groups of 128                 8.5 / 7.1 / 9.9
//   12 groups of 512                   - /  17 /  14
//   64 groups of 128                  34 /  22 /  24
//   64 groups of 256                  58 /  34 /  31
// The few-rows form therefore for groups of at most 32 rows, or where its
// small tiles number at most 2.6 per CU; else 128x128 tiles until they number
// 1.3 per CU and groups hold 192 rows.  Groups that fill whole tiles count half
// a tile too many: 4 groups of 256 and 12 of 64 above (684 tiles by the count,
// the limit is 665) take 128x128 tiles, 18 and 15% slower.  And where most groups are
// empty, `full` is far from the groups with rows: a few long groups among many
// empty ones can take the few-rows form, up to 1.7 times the best one's time.
inline GemmForm gemm_form(const GroupedGemmArgs &a, int cus) {
    const int64_t full = full_groups(a.M, a.groups);
    const auto tiles = [&](int bm, int bn) { return (a.M + bm * full / 2) / bm * cdiv(a.N, bn); };
    const bool few_fits = max_tiles(a.M, a.groups, kFewM) * cdiv(a.N, kFewN) < 2 * kMaxBlocks;   // of 256 threads
    if (few_fits && (a.M <= 32 * full || 10 * tiles(kFewM, kFewN) <= 26 * cus)) return GemmForm::kFewRows;
    if (10 * tiles(128, 128) <= 13 * cus || a.M < 192 * full) return GemmForm::kTiles128;
    const int64_t bytes = padded(a.K) / 2;
    if (cus > 0 && a.K > 0 &&
        stream_fits(a, (a.M + 15 * full) / 16 * 16 * bytes, a.groups * (cdiv(a.N, 16) * 16) * bytes))
        return GemmForm::kPersistent;
    return GemmForm::kTiles256;
}

// 128x128 tiles while they number at most 1.3 per CU: 4 groups of 1200 x 1024
// 6.8 us (persistent 8.3), 12 groups of it 12.8 (10.8).
inline GemmForm wgrad_form(const GroupedGemmArgs &a, int cus) {
    if (10 * a.groups * cdiv(a.N, 128) * cdiv(a.K, 128) <= 13 * cus) return GemmForm::kTiles128;
    const int64_t bytes = (a.M + 127 * full_groups(a.M, a.groups)) / 128 * 64;   // a blob's per row
    if (cus > 0 && stream_fits(a, cdiv(a.N, 16) * 16 * bytes, cdiv(a.K, 16) * 16 * bytes))
        return GemmForm::kPersistent;
    return GemmForm::kTiles256;
}

}  // namespace mx
