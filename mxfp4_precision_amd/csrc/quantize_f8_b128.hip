// FP8 quantization of bf16 with one E8M0 scale for each block of 128 elements:
// row-wise (blocks along N), column-wise (the transpose, blocks along M) or
// both from one read, either with 128 x 128 tiles that share one scale.
//
// scale byte c: the smallest with amax <= MAX 2^(c - 127), MAX = 448 (E4M3) or
// 57344 (E5M2), so nothing saturates; 0xFF for a block that holds Inf or NaN.
// code = x 2^(127 - c) rounded to nearest even (V_CVT_SCALEF32_PK_FP8_BF16 and
// its E5M2 form: two elements an instruction, straight from bf16).
//
// A workgroup takes a 128 x 128 tile: a thread 4 consecutive rows x 16
// columns.  A row's maximum is found in the 8 lanes that hold it, a column's in
// a wave by lane exchanges and across the four waves in LDS.  Both blobs' codes
// go through LDS (16-byte chunks, swizzled so that 8 lanes touch all banks), so
// that each wave stores whole 1 KB atoms.
//
// Bound by memory.  Measured on MI355X, in turn: 16384 x 4096 both directions
// 49.2 us, 5.5 TB/s (54 with cached stores), row-wise 36.5, column-wise 37.9;
// 4096 x 4096 11.6 (14.5 with cached stores); 333 x 1000 5.6.  Non-temporal
// loads: 16384 x 4096 both directions 57.

#include "f8_b128.h"

namespace mx {
namespace {

constexpr int kTile = 128;

// Byte offset of the 16 codes (row r, elements k .. k + 15) in a blob.
template <int LAYOUT>
__device__ __forceinline__ int64_t data_at(int64_t r, int64_t k, int64_t Lp) {
    if constexpr (LAYOUT == MX_LAYOUT_TILED)
        return ((r >> 4) * (Lp / 64) + (k >> 6)) * 1024 + ((r & 15) + 16 * ((k & 63) >> 4)) * 16;
    else
        return r * Lp + k;
}

// One row's scale byte for block kb (of nb), and zeros for the slots behind
// the last block of its scale word.
template <int LAYOUT>
__device__ __forceinline__ void store_scale(uint8_t *s, int64_t r, int64_t kb, int64_t nb, uint32_t c) {
    if constexpr (LAYOUT == MX_LAYOUT_TILED) {
        uint8_t *word = s + ((r >> 4) * cdiv(nb, 4) + (kb >> 2)) * 64 + (r & 15) * 4;
        word[kb & 3] = (uint8_t)c;
        if (kb == nb - 1)
#pragma unroll
            for (int e = 1; e < 4; ++e)
                if (e > (int)(kb & 3)) word[e] = 0;
    } else {
        s[r * nb + kb] = (uint8_t)c;
    }
}

// FR, FC: formats of the row-wise and the column-wise blob, or -1: not wanted.
template <int LAYOUT, int FR, int FC>
__global__ __launch_bounds__(256) void quantize_f8_b128_kernel(F8QuantArgs a, uint32_t tiles_n) {
    __shared__ u4_t s_code[FR >= 0 && FC >= 0 ? 2 : 1][1024];   // 128 blob rows x 8 chunks of 16 codes
    __shared__ uint32_t s_col[4][64];        // a wave's column maxima, two a word
    __shared__ __attribute__((aligned(16))) uint8_t s_scale[2][kTile];    // scale bytes of the tile's rows and columns
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int tr = t >> 3, tc = t & 7;
    const uint32_t tm = blockIdx.x / tiles_n, tn = blockIdx.x - tm * tiles_n;
    const int64_t r0 = (int64_t)tm * kTile, c0 = (int64_t)tn * kTile;
    const bool need_tile = (FR >= 0 && a.row_2d) || FC >= 0;

    u4_t v[4][2];
    if (r0 + kTile <= a.M && c0 + kTile <= a.N) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const u4_t *p = reinterpret_cast<const u4_t *>(a.x + (r0 + 4 * tr + i) * a.ldx + c0 + 16 * tc);
            v[i][0] = p[0];
            v[i][1] = p[1];
        }
    } else if (a.ldx < (int64_t(1) << 22)) {
        // at the edges through a range-checked buffer that ends with the tensor (in
        // whole words, which is what the check goes by), without branches: rows past
        // it read 0, and what lies between the rows is masked
        const int64_t rows = a.M - r0 < kTile ? a.M - r0 : kTile;
        const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t *>(a.x + r0 * a.ldx + c0), (short)0,
            (int)((((rows - 1) * a.ldx + (a.N - c0)) * 2 + 3) & ~int64_t(3)), 0x00020000);
        const int left = (int)(a.N - c0 < kTile ? a.N - c0 : kTile) - 16 * tc;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int off = ((4 * tr + i) * (int)a.ldx + 16 * tc) * 2;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v[i][h] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rx, off + 16 * h, 0, 0));
            }
        }
        uint32_t keep[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) keep[w] = (2 * w < left ? 0x0000FFFFu : 0u) | (2 * w + 1 < left ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int w = 0; w < 8; ++w) v[i][w >> 2][w & 3] &= keep[w];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) load16(a.x, a.M, a.N, a.ldx, r0 + 4 * tr + i, c0 + 16 * tc, v[i]);
    }

    uint32_t row_max[4];
    uint32_t cm[8];
#pragma unroll
    for (int w = 0; w < 8; ++w) cm[w] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const uint32_t p = v[i][w >> 2][w & 3] & 0x7FFF7FFFu;
            m = max2(m, p);
            cm[w] = max2(cm[w], p);
        }
        m = max2_dpp<0xB1>(m);    // lanes ^ 1
        m = max2_dpp<0x4E>(m);    // lanes ^ 2
        m = max2_dpp<0x141>(m);   // mirrored in 8 lanes
        row_max[i] = (m & 0xFFFFu) > (m >> 16) ? (m & 0xFFFFu) : (m >> 16);
    }
    uint32_t tile_max = 0;
    if (need_tile) {
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            cm[w] = max2_dpp<0x128>(cm[w]);   // lanes rotated by 8 in 16
            cm[w] = max2_xor<16>(cm[w]);
            cm[w] = max2_xor<32>(cm[w]);
        }
        if (lane < 8) {
            *reinterpret_cast<u4_t *>(&s_col[wave][8 * tc]) = u4_t{cm[0], cm[1], cm[2], cm[3]};
            *reinterpret_cast<u4_t *>(&s_col[wave][8 * tc + 4]) = u4_t{cm[4], cm[5], cm[6], cm[7]};
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u4_t m = *reinterpret_cast<const u4_t *>(&s_col[0][8 * tc + 4 * h]);
#pragma unroll
            for (int w = 1; w < 4; ++w) {
                const u4_t q = *reinterpret_cast<const u4_t *>(&s_col[w][8 * tc + 4 * h]);
#pragma unroll
                for (int e = 0; e < 4; ++e) m[e] = max2(m[e], q[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) cm[4 * h + e] = m[e];
        }
        if (a.row_2d || a.col_2d) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) m = max2(m, cm[w]);
            m = max2_dpp<0xB1>(m);
            m = max2_dpp<0x4E>(m);
            m = max2_dpp<0x141>(m);
            tile_max = (m & 0xFFFFu) > (m >> 16) ? (m & 0xFFFFu) : (m >> 16);
        }
    }

    // Row-wise: chunk tc of row r at 8 r + (tc ^ r % 8).
    if constexpr (FR >= 0) {
        uint32_t bytes = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * tr + i;
            const uint32_t c = scale_byte<FR>(a.row_2d ? tile_max : row_max[i]);
            const float scale = scale_of(c);
            u4_t q;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                q[e] = encode4<FR>(v[i][e >> 1][(e & 1) * 2], v[i][e >> 1][(e & 1) * 2 + 1], scale);
            if (c == 0xFFu) q = u4_t{};
            s_code[0][8 * r + (tc ^ (r & 7))] = q;
            bytes |= (r0 + r < a.M ? c : 0u) << (8 * i);   // rows past the tensor: zero bytes
        }
        if (tc == 0) reinterpret_cast<uint32_t *>(s_scale[0])[tr] = bytes;
    }
    // Column-wise: of column j, rows 16 h .. 16 h + 15 are chunk h, at 8 j +
    // (h ^ j % 8 ^ j / 16); the thread's 4 rows are one word of it.
    if constexpr (FC >= 0) {
        u4_t bytes = {};
        uint32_t *words = reinterpret_cast<uint32_t *>(&s_code[FR >= 0 ? 1 : 0][0]);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int j = 16 * tc + e;
            const uint32_t c = scale_byte<FC>(a.col_2d ? tile_max : (cm[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
            // rows i and i + 1 of column j in one word
            const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
            const uint32_t w01 = __builtin_amdgcn_perm(v[1][e >> 3][(e & 7) >> 1], v[0][e >> 3][(e & 7) >> 1], sel);
            const uint32_t w23 = __builtin_amdgcn_perm(v[3][e >> 3][(e & 7) >> 1], v[2][e >> 3][(e & 7) >> 1], sel);
            uint32_t q = encode4<FC>(w01, w23, scale_of(c));
            if (c == 0xFFu) q = 0u;
            words[4 * (8 * j + ((tr >> 2) ^ (j & 7) ^ tc)) + (tr & 3)] = q;
            bytes[e >> 2] |= (c0 + j < a.N ? c : 0u) << (8 * (e & 3));
        }
        if (tr == 0) reinterpret_cast<u4_t *>(s_scale[1])[tc] = bytes;
    }
    __syncthreads();
    if constexpr (FR >= 0) {
        const int64_t R16 = LAYOUT == MX_LAYOUT_TILED ? cdiv(a.M, 16) * 16 : a.M;
        if (t < kTile && r0 + t < R16)
            store_scale<LAYOUT>(a.s_row, r0 + t, tn, cdiv(a.N, kTile), s_scale[0][t]);
    }
    if constexpr (FC >= 0) {
        const int64_t R16 = LAYOUT == MX_LAYOUT_TILED ? cdiv(a.N, 16) * 16 : a.N;
        const int j = t & (kTile - 1);
        if (t >= kTile && c0 + j < R16)
            store_scale<LAYOUT>(a.s_col, c0 + j, tm, cdiv(a.M, kTile), s_scale[1][j]);
    }
    // Each wave stores atoms: 16 rows x 4 chunks.
    const int ar = lane & 15, ac = lane >> 4;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const int atom = 4 * n + wave, g = atom >> 1, r = 16 * g + ar, h = 4 * (atom & 1) + ac;
        if constexpr (FR >= 0) {
            const int64_t R16 = LAYOUT == MX_LAYOUT_TILED ? cdiv(a.M, 16) * 16 : a.M;
            if (r0 + r < R16)
                __builtin_nontemporal_store(
                    s_code[0][8 * r + (h ^ (r & 7))],
                    reinterpret_cast<u4_t *>(a.q_row + data_at<LAYOUT>(r0 + r, c0 + 16 * h, padded(a.N))));
        }
        if constexpr (FC >= 0) {
            const int64_t R16 = LAYOUT == MX_LAYOUT_TILED ? cdiv(a.N, 16) * 16 : a.N;
            if (c0 + r < R16)
                __builtin_nontemporal_store(
                    s_code[FR >= 0 ? 1 : 0][8 * r + (h ^ (r & 7) ^ g)],
                    reinterpret_cast<u4_t *>(a.q_col + data_at<LAYOUT>(c0 + r, r0 + 16 * h, padded(a.M))));
        }
    }
}

template <int FR, int FC>
hipError_t launch_pair(const F8QuantArgs &a, mx_layout layout, hipStream_t stream) {
    const int64_t tiles_n = cdiv(a.N, kTile);
    const dim3 grid((unsigned)(tiles_n * cdiv(a.M, kTile)));
    if (layout == MX_LAYOUT_TILED)
        hipLaunchKernelGGL((quantize_f8_b128_kernel<MX_LAYOUT_TILED, FR, FC>), grid, dim3(256), 0, stream, a, (uint32_t)tiles_n);
    else
        hipLaunchKernelGGL((quantize_f8_b128_kernel<MX_LAYOUT_CANONICAL, FR, FC>), grid, dim3(256), 0, stream, a,
                           (uint32_t)tiles_n);
    return hipGetLastError();
}

template <int FR>
hipError_t launch_row(const F8QuantArgs &a, mx_layout layout, hipStream_t stream) {
    if (!a.q_col) {
        if constexpr (FR >= 0) return launch_pair<FR, -1>(a, layout, stream);
        else return hipErrorInvalidValue;
    }
    return a.fmt_col == MX_FP8_E4M3 ? launch_pair<FR, MX_FP8_E4M3>(a, layout, stream)
                                    : launch_pair<FR, MX_FP8_E5M2>(a, layout, stream);
}

}  // namespace

hipError_t launch_quantize_f8_b128(const F8QuantArgs &a, mx_layout layout, hipStream_t stream) {
    if (!a.q_row) return launch_row<-1>(a, layout, stream);
    return a.fmt_row == MX_FP8_E4M3 ? launch_row<MX_FP8_E4M3>(a, layout, stream)
                                    : launch_row<MX_FP8_E5M2>(a, layout, stream);
}

}  // namespace mx
