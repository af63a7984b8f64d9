// Which kernel form an FP8 product with block scales takes: arithmetic on the
// call's sizes on the host.  `cus`: compute units of the device, 0 if unknown.
#pragma once

#include "mx_internal.h"

namespace mx {

enum class F8Form {
    kFewRows,    // operands straight from memory to registers
    kTiles128,   // one 128x128 tile per workgroup
    kPersistent, // one workgroup per CU, 256x256 tiles
    kTiles256    // one 256x256 tile per workgroup
};

// Whether the persistent form's epilogue takes the output: bf16, whole 16-byte
// chunks, 32-bit offsets.
inline bool f8_persistent_fits(const F8GemmArgs &a) {
    return a.out_dtype == MX_BF16 && a.N % 8 == 0 && a.ldc <= ((int64_t(1) << 30) - 1) / a.M;
}

// Measured on MI355X in us, few rows / 128x128 / persistent / 256x256:
//    333 x  4096 x 4096   15.1 / 16.6 / 48 / 40      768 few-rows tiles
//    512 x  4096 x 4096   19.8 / 17.6 / 53 / 39      1024
//    256 x  8192 x 1024    7.6 /  7.2 / 20 / 18      1024
//    192 x  8192 x 1024    6.5 /  7.3 / 19 / 19      768
//   1024 x  1024 x 8192   20.8 / 29.9 / 89 / 67      512
//   2048 x  4096 x 4096     69 / 32.2 / 54 / 45      2 tiles of 128x128 per CU
//   4096 x  2880 x 2880      - / 37.0 / 41.9 / 39.3  2.9
//   1536 x  8192 x 1024     30 / 24.4 / 20.3 / 21.7  3
//   4096 x  4096 x 4096      - / 62.2 / 53.4 / 57.7  4
// The few-rows form therefore up to 3 of its tiles per CU.  Two 128x128 tiles run
// on a CU at a time, and their time goes by their number, 3.3 for each tile a CU
// where a round of 256x256 tiles takes 10 and a part of one as long: 128x128
// tiles where that is less, which is also where a last round of 256x256 ones
// would leave most CUs idle.  The persistent form's K-loop ends at a multiple of
// 512; 8192 x 8192, 128x128 / persistent / 256x256: K 512 65 / 54 / 69, 640 70 / 69 /
// 74, 768 75 / 70 / 78, 1024 84 / 72 / 89, 1152 92 / 89 / 94, 1280 98 / 91 / 99, so K
// does not decide.  These are bf16 outputs.  fp32, 128x128 / 256x256: 4096 x 4096 x
// 16384 271 / 203 (persistent with bf16: 191), 8192 x 8192 x 1024 131 / 155: where
// stores of fp32 outweigh a short K, smaller tiles would be faster than the rule's.
inline F8Form f8_gemm_form(const F8GemmArgs &a, int cus) {
    const auto tiles = [&](int bm, int bn) { return cdiv(a.M, bm) * cdiv(a.N, bn); };
    if (a.M <= 64 || tiles(64, 32) <= 3 * (int64_t)cus) return F8Form::kFewRows;
    const int64_t rounds = cus > 0 ? cdiv(tiles(256, 256), cus) : 0;
    if (33 * tiles(128, 128) < 100 * rounds * cus) return F8Form::kTiles128;
    return cus > 0 && f8_persistent_fits(a) ? F8Form::kPersistent : F8Form::kTiles256;
}

// Whether a linear layer of M rows quantizes x inside the product, where every
// workgroup reads and quantizes 16 rows for 16 columns.  In us, one launch / two, in
// a captured run over other weights each time (K -> N; from 17 rows with a grid of
// one more row tile for every 16):
//                1 row         8          16          17          32          64
//   1024 -> 1024  2.8 / 5.4   3.1 / 5.4   3.5 / 5.4   3.5 / 6.0   3.5 / 6.1   3.6 / 6.9
//   4096 -> 4096  6.9 / 8.8   7.4 / 8.9   8.4 / 9.1  11.8 / 11.9 12.3 / 12.1 20.2 / 13.0
//   2889 -> 5003  8.6 / 9.3   9.0 / 9.4  10.7 / 9.5  12.2 / 10.3 15.4 / 10.4 21.2 / 11.5
//   8192 -> 2048  8.9 / 11.4  9.8 / 11.5 12.3 / 11.5 11.8 / 17.4 12.0 / 17.4 20.5 / 19.5
//   4096 -> 8192  9.9 / 11.9 10.9 / 12.0 13.2 / 12.0 19.9 / 13.6 20.8 / 13.7 36.5 / 15.2
inline bool f8_linear_fused(int64_t M) { return M <= 16; }

// Workgroups of the largest grid (of 256 threads: fewer than 2^32 threads).
constexpr int64_t kF8MaxBlocks = int64_t(1) << 23;

// Whether every form's grid holds the product.  (The few-rows form takes at
// most 64 rows, or few tiles; its N is below 2^24, as B is below 2 GiB.)
inline bool f8_gemm_fits(int64_t M, int64_t N) {
    return cdiv(M, 128) == 0 || cdiv(N, 128) <= (kF8MaxBlocks - 1) / cdiv(M, 128);
}

}  // namespace mx
