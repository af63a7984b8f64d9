// Device side of FP8 with block scales of 128: scale bytes, codes and the loads
// of ragged rows, shared by the quantizer and the linear layer of few rows.
#pragma once

#include "mx_internal.h"

namespace mx {
namespace {

typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef unsigned short us2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
typedef short s2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {   // of two 16-bit patterns each
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2_t, a),
                                                                  __builtin_bit_cast(us2_t, b)));
}
template <int CTRL>
__device__ __forceinline__ uint32_t max2_dpp(uint32_t v) {
    return max2(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
// Largest pattern of the lanes that differ in bit 4 (16) or 5 (32) of their
// number: the swap of a register's odd rows with its own even ones leaves each
// pair's values in two registers, without LDS.
template <int MASK>
__device__ __forceinline__ uint32_t max2_xor(uint32_t v) {
    static_assert(MASK == 16 || MASK == 32, "");
    if constexpr (MASK == 16) {
        const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return max2(p[0], p[1]);
    } else {
        const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return max2(p[0], p[1]);
    }
}

// Scale byte of a block from its largest bf16 magnitude: the exponent field
// less the format's, one more when the mantissa is above 1.75 (the carry of the
// addition).
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    if (amax >= 0x7F80u) return 0xFFu;
    const int c = (int)((amax + 0x1Fu) >> 7) - (FMT == MX_FP8_E4M3 ? 8 : 15);
    return c > 0 ? (uint32_t)c : 0u;
}

// The number 2^(c - 127) that the conversions divide by.
__device__ __forceinline__ float scale_of(uint32_t c) {
    return __uint_as_float(c ? c << 23 : 0x00400000u);
}

// Two bf16 elements of a word to two codes in the low (HI: high) half of `old`.
template <int FMT, bool HI>
__device__ __forceinline__ uint32_t encode2(uint32_t old, uint32_t w, float scale) {
    const s2_t o = __builtin_bit_cast(s2_t, old);
    const bf2_t v = __builtin_bit_cast(bf2_t, w);
    if constexpr (FMT == MX_FP8_E4M3)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, v, scale, HI));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(o, v, scale, HI));
}
template <int FMT>
__device__ __forceinline__ uint32_t encode4(uint32_t w0, uint32_t w1, float scale) {
    return encode2<FMT, true>(encode2<FMT, false>(0u, w0, scale), w1, scale);
}

// 16 elements of row r from column j0: 0 outside the tensor.  A chunk of 8 in
// which the row ends is read whole where another row follows (ldx is a multiple
// of 8, so the chunk lies inside the row's stride) and by elements in the last
// row, behind which the tensor may end; what is past N is masked.
__device__ __forceinline__ void load16(const uint16_t *__restrict__ x, int64_t M, int64_t N, int64_t ldx, int64_t r,
                                       int64_t j0, u4_t (&v)[2]) {
    v[0] = v[1] = u4_t{};
    if (r >= M) return;
    const uint16_t *p = x + r * ldx + j0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t left = N - (j0 + 8 * h);   // elements from here to the row's end
        if (left >= 8 || (left > 0 && r + 1 < M)) {
            v[h] = *reinterpret_cast<const u4_t *>(p + 8 * h);
        } else if (left > 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {   // (all loads at once: past the end the last element again)
                const uint32_t b = p[8 * h + (e < left ? e : (int)left - 1)];
                v[h][e >> 1] |= b << (16 * (e & 1));
            }
        }
        if (left < 8)
#pragma unroll
            for (int w = 0; w < 4; ++w)
                v[h][w] &= (2 * w < left ? 0x0000FFFFu : 0u) | (2 * w + 1 < left ? 0xFFFF0000u : 0u);
    }
}

}  // namespace
}  // namespace mx
