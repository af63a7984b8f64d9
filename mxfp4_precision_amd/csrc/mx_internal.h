// Internal declarations shared by the libmxfp4 translation units (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mxfp4.h"

namespace mx {

constexpr int64_t kBlock = 32;   // elements per scale block
constexpr int64_t kPad = 128;    // quantized-axis padding

__host__ __device__ inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
__host__ __device__ inline int64_t padded(int64_t n) { return cdiv(n, kPad) * kPad; }

// Per-direction options in the form the kernels take them.
struct DirOpts {
    uint32_t use_2d;
    uint32_t use_sr;
    uint32_t key0, key1;        // Philox key = seed
    uint32_t tensor_id;
    uint64_t index_base;
    uint32_t rht;               // random Hadamard transform seed, 0 = off
    uint32_t fmt;               // MXFP6 element format (2 = E2M3, 3 = E3M2); unused for MXFP4
};

struct QuantArgs {
    const uint16_t *x;
    int64_t M, N, ldx;
    const uint16_t *g;          // second factor of the multiply prologue (same shape), or NULL
    int64_t ldg;
    int64_t M_pad, N_pad;       // padded quantized axes (col blob, row blob)
    DirOpts row, col;
    uint32_t sr_pairs;          // 1: N and both index bases are multiples of 16
    uint8_t *q_row, *s_row, *q_col, *s_col;
    int64_t row_tile0;          // first 128-row tile of this launch (set by the launchers)
    // grouped quantization: cumulative row ends of the groups and, optionally,
    // the row of x (x_rows of them) that each grouped row is
    const int32_t *ends, *row_index;
    int32_t groups;
    int64_t x_rows;
};

constexpr int kXcds = 8;   // dies of the chip, each with an L2 of its own; workgroups go to them round-robin

struct GroupedGemmArgs {
    const int32_t *ends;        // cumulative row ends of the groups, device memory
    int groups;
    int64_t M, N, K;            // M: rows of all groups
    const uint8_t *A, *As, *B, *Bs;
    const uint16_t *bias;       // groups x N, or NULL
    mx_dtype out_dtype;
    void *C;
    int64_t ldc, group_stride;
};

// FP8 with a scale for each block of 128.
struct F8QuantArgs {
    const uint16_t *x;
    int64_t M, N, ldx;
    int fmt_row, fmt_col;       // mx_fp8_format
    bool row_2d, col_2d;        // 128 x 128 tiles share a scale
    uint8_t *q_row, *s_row, *q_col, *s_col;   // either pair may be NULL
};
struct F8GemmArgs {
    int64_t M, N, K;
    int fmt_a, fmt_b;
    const uint8_t *A, *As, *B, *Bs;
    const uint16_t *bias;       // N, or NULL
    mx_dtype out_dtype;
    void *C;
    int64_t ldc;
};
// mx_linear_f8_b128: the A of the product is x, quantized on the way.
struct F8LinearArgs {
    const uint16_t *x;
    int64_t ldx;
    F8GemmArgs g;               // A, As: the workspace's blob, if the form needs one
};

// A layer of experts for a few tokens.
constexpr int kExpertTokens = 64, kExpertTopk = 32, kExpertsMost = 1024;
constexpr int kExpertSplits = 256;   // most workgroups of the down product where it is split
struct ExpertsArgs {
    int tokens, experts, topk;
    int64_t K, inner, ldx, ldy;
    const uint16_t *x;
    const int32_t *ids;
    const float *weights;
    const uint8_t *W1, *W1s, *W2, *W2s;
    void *y;
    int *counters;              // kExpertSplits, zeroed by the first kernel
    float *sums;                // kExpertSplits x 16 x tokens
    uint16_t *h;                // expert_tiles x 16 x padded(inner) activations, two bf16 each
};
// Column tiles of 16 tokens that pairs can make: one for each expert that they
// name, and one more for every 16.
inline int64_t expert_tiles(int64_t pairs) { return (pairs < kExpertsMost ? pairs : kExpertsMost) + pairs / 16; }
// Tiles of 16 rows of the up product that a workgroup takes.  Two halve the reading
// of activations and the workgroups that find out the routing, but need 4 workgroups
// of one tile for each CU, for all experts that the pairs can name.  In us a call,
// one / two, after that number of workgroups: 360 (5 tokens, 2 of 9, 1001 x 523)
// 12.9 / 13.9; 512 (1 token, 8 of 64, 2048 x 1024 17.9 / 19.4; 64 tokens, 8 of 8,
// 2048 x 1024 40.7 / 44.2); 768 (3 tokens, 4 of 64, 2048 x 1024) 20.1 / 22.1; 1024 (2
// tokens, 8 of 64, 2048 x 1024 25.9 / 25.2; 1 token, 1 of 8, 4096 x 16384 33.0 / 31.1;
// 2 tokens, 2 of 8, 2048 x 4096 23.2 / 24.2); 4096 (64 tokens, 8 of 64, 2048 x 1024)
// 87.5 / 81.3; 5888 (16 tokens, 4 of 32, 2880 x 2880) 79.6 / 74.4; 8192 (64 tokens, 8
// of 256, 1024 x 512) 65.6 / 53.0.
inline int expert_row_tiles(int slots, int64_t inner) { return slots * (padded(inner) / 16) >= 1024 ? 2 : 1; }
// Workgroups that share a row tile of the down product: one workgroup per CU in all,
// each with four atoms for each of its 8 waves at least.  In us a call, one per CU /
// 1.5: 160 row tiles (K 2560, inner 768), 64 tokens, 8 of 128 110.5 / 110.5, 8 tokens
// 40.1 / 41.2; 128 (2048 x 1024, 8 of 64), 64 tokens 77.4 / 81.3, 16 tokens 43.5 /
// 46.5, 2 tokens 24.9 / 25.9; 96 (1536 x 1024, 6 of 64), 16 tokens 36.3 / 36.3; 64
// (1024 x 4096, 4 of 16), 64 tokens 70.3 / 72.3; 48 (768 x 2048, 4 of 16), 8 tokens
// 23.4 / 24.7; 32 (512 x 4096, 2 of 8), 8 tokens 20.8 / 22.4, with half as many as one
// per CU 19.8.  Not split at all, 128 row tiles: 64 tokens 93.7, 1 token 17.1 against
// 17.6.
inline int expert_splits(int slots, int64_t tiles, int64_t inner) {
    const int64_t atoms = slots * (padded(inner) / 128);
    int64_t n = atoms / 32;
    if (n > kExpertSplits / tiles) n = kExpertSplits / tiles;
    return n > 1 ? (int)n : 1;
}

// Descriptors of one AdamW launch, passed as kernel arguments.
struct AdamwItem {
    void *param;
    const void *grad;
    void *m, *v;
    uint8_t *ms, *vs;           // block scales of 8-bit states
    void *copy;                 // bf16 copy of the parameters, or NULL
    int64_t numel;
    uint32_t chunk_end;         // workgroups of this and the items before it
    uint32_t tensor_id;
};
constexpr int kAdamwItems = 48;
// One launch's kernel arguments.  They are copied for each launch, so a few
// tensors go with a short table.
template <int ITEMS>
struct AdamwTable {
    int count;
    float beta1, one_minus_beta1, beta2, one_minus_beta2, eps;
    mx_adamw_step step;
    const mx_adamw_step *dev_step;
    AdamwItem t[ITEMS];
};
using AdamwBatch = AdamwTable<kAdamwItems>;
static_assert(sizeof(AdamwBatch) <= 4000, "kernel arguments");

// Gradients of one launch, passed as kernel arguments.
struct GradItem {
    void *g;
    int64_t numel;
    uint32_t chunk_end;         // workgroups of this and the items before it
    uint32_t f32;               // 1: fp32, 0: bf16
};
constexpr int kGradItems = 96, kGradFew = 8;
template <int ITEMS>
struct GradTable {
    int64_t chunk;              // elements of a workgroup, a multiple of 8
    int count;
    GradItem t[ITEMS];
};
using GradBatch = GradTable<kGradItems>;
static_assert(sizeof(GradBatch) <= 4000, "kernel arguments");
struct GradNormOut {
    double max_norm, grad_scale;
    mx_grad_norm_info *info;
    mx_adamw_step *step;        // or NULL
};
// The norm's chunks: all tensors make kGradChunks of them at most, and one more
// for each tensor.
constexpr int64_t kGradChunks = 2048;
inline int64_t grad_chunk(int64_t total) {
    const int64_t even = cdiv(cdiv(total, kGradChunks), 8) * 8;
    return even > 8192 ? even : 8192;
}
constexpr int64_t kScaleChunk = 8192;       // elements that a workgroup scales
// Elements of up to kGradFew tensors that one workgroup sums, a wave each.  fp32, one
// launch / two in us: 4 of 1000 2.7 / 4.5, 8 of 2048 2.7 / 5.0, one of 4096 2.7 / 4.2, of
// 8192 3.3 / 4.4, of 16384 4.7 / 4.6.
constexpr int64_t kGradFewTotal = 16384;

// Grid dimension y of one launch holds at most 65536 workgroups on gfx950
// (hipDeviceAttributeMaxGridDimY); the quantize launchers cover taller inputs
// with several launches of kMaxRowTiles row tiles each.
constexpr int64_t kMaxRowTiles = 65535;

// Kernel launchers (quantize.hip, gemm.hip, convert.hip, dequantize.hip).  They assume validated arguments.
hipError_t launch_quantize(const QuantArgs &a, bool dual, mx_layout layout, hipStream_t stream);
hipError_t launch_quantize_fp6(const QuantArgs &a, bool dual, mx_layout layout, hipStream_t stream);
hipError_t launch_quantize_mul(const QuantArgs &a, bool dual, mx_layout layout, hipStream_t stream);
hipError_t launch_gemm_fp6(int64_t M, int64_t N, int64_t K, int fmt_a, const uint8_t *A, const uint8_t *As,
                           int fmt_b, const uint8_t *B, const uint8_t *Bs, mx_dtype out_dtype, void *C, int64_t ldc,
                           hipStream_t stream);
hipError_t launch_gemm(int64_t M, int64_t N, int64_t K, const uint8_t *A, const uint8_t *As,
                       const uint8_t *B, const uint8_t *Bs, const uint16_t *bias, mx_dtype out_dtype, void *C,
                       int64_t ldc, hipStream_t stream);
int device_cu_count();   // compute units of the current device (cached), 0 if unknown
hipError_t launch_gemm_fp8(int64_t M, int64_t N, int64_t K, const uint8_t *A, const float *a_scale_inv,
                           const uint8_t *B, const float *b_scale_inv, mx_dtype out_dtype, void *C, int64_t ldc,
                           hipStream_t stream);
hipError_t launch_quantize_fp8(const uint16_t *x, int64_t M, int64_t N, int64_t ldx, mx_layout layout,
                               uint8_t *q_row, uint8_t *q_col, float *info, hipStream_t stream);
hipError_t launch_quantize_f8_b128(const F8QuantArgs &a, mx_layout layout, hipStream_t stream);
hipError_t launch_gemm_f8_b128(const F8GemmArgs &a, hipStream_t stream);
hipError_t launch_linear_f8_b128(const F8LinearArgs &a, hipStream_t stream);
hipError_t launch_layout_convert(bool to_tiled, int64_t rows, int64_t length, const uint8_t *q_src,
                                 const uint8_t *s_src, uint8_t *q_dst, uint8_t *s_dst, hipStream_t stream);
hipError_t launch_quantize_grouped(const QuantArgs &a, bool dual, hipStream_t stream);
hipError_t launch_gemm_grouped(const GroupedGemmArgs &a, hipStream_t stream);
hipError_t launch_gemm_grouped_wgrad(const GroupedGemmArgs &a, hipStream_t stream);
int64_t adamw_chunks(int64_t numel);   // workgroups that numel elements take
hipError_t launch_adamw(const AdamwBatch &b, bool p32, bool g32, bool s8, bool sr, hipStream_t stream);
hipError_t launch_experts(const ExpertsArgs &a, mx_dtype out_dtype, hipStream_t stream);
hipError_t launch_grad_sums(const GradBatch &b, double *sums, hipStream_t stream);
hipError_t launch_grad_norm(const double *sums, int n, const GradNormOut &o, hipStream_t stream);
hipError_t launch_grad_norm_few(const GradBatch &b, const GradNormOut &o, hipStream_t stream);
hipError_t launch_grad_finish(const GradNormOut &o, hipStream_t stream);
hipError_t launch_grad_scale(const GradBatch &b, const mx_grad_norm_info *info, hipStream_t stream);
hipError_t launch_dequantize(const uint8_t *q, const uint8_t *s, int64_t rows, int64_t length,
                             mx_layout layout, float *out, int64_t ldo, hipStream_t stream);
hipError_t launch_measure_mfma(int fmt_a, int fmt_b, const void *ops, int workgroups, int64_t iters, float *out,
                               hipStream_t stream);

}  // namespace mx
