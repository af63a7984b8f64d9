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

inline F8Form f8_gemm_form(const F8GemmArgs &a, int cus) {
    const auto tiles = [&](int bm, int bn) { return cdiv(a.M, bm) * cdiv(a.N, bn); };
    if (a.M <= 64 || 10 * tiles(64, 32) <= 26 * (int64_t)cus) return F8Form::kFewRows;
    if (10 * tiles(128, 128) <= 13 * (int64_t)cus) return F8Form::kTiles128;
    if (cus > 0 && a.out_dtype == MX_BF16 && a.N % 8 == 0 && tiles(256, 256) > cus &&
        a.M * a.ldc * 2 < (int64_t(1) << 31))
        return F8Form::kPersistent;
    return F8Form::kTiles256;
}

// Whether a linear layer of M rows quantizes x inside the product.  In us, one
// launch / two: 1 row, 4096 x 4096 7.7 / 10.9; 23 rows (two row tiles), 5003 x
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
