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
// would leave most CUs idle.
inline F8Form f8_gemm_form(const F8GemmArgs &a, int cus) {
    const auto tiles = [&](int bm, int bn) { return cdiv(a.M, bm) * cdiv(a.N, bn); };
    if (a.M <= 64 || tiles(64, 32) <= 3 * (int64_t)cus) return F8Form::kFewRows;
    const int64_t rounds = cus > 0 ? cdiv(tiles(256, 256), cus) : 0;
    if (33 * tiles(128, 128) < 100 * rounds * cus) return F8Form::kTiles128;
    return cus > 0 && f8_persistent_fits(a) ? F8Form::kPersistent : F8Form::kTiles256;
}

// Whether a linear layer of M rows quantizes x inside the product.  In us, one
// launch / two: 1 row, 4096 x 4096 5.9 / 10; 23 rows (two row tiles), 5003 x
// 2889 14.1 / 11.7, as every workgroup reads and quantizes all of x.
inline bool f8_linear_fused(int64_t M) { return M <= 16; }

// Workgroups of the largest grid (of 256 threads: fewer than 2^32 threads).
constexpr int64_t kF8MaxBlocks = int64_t(1) << 23;

// Whether every form's grid holds the product.  (The few-rows form takes at
// most 64 rows, or few tiles; its N is below 2^24, as B is below 2 GiB.)
inline bool f8_gemm_fits(int64_t M, int64_t N) {
    return cdiv(M, 128) == 0 || cdiv(N, 128) <= (kF8MaxBlocks - 1) / cdiv(M, 128);
}

}  // namespace mx
