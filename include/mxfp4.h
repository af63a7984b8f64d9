/*
 * mxfp4.h -- C ABI of libmxfp4: MXFP4 block quantization of bf16 tensors and
 * the block-scaled FP4 x FP4 ("a4w4") GEMM that consumes the blobs, for
 * MI355X (gfx950).
 *
 * Formats follow the OCP Microscaling Formats (MX) Specification v1.0:
 * 32-element blocks, one E8M0 scale byte per block (2^(byte-127), 0xFF = NaN)
 * and E2M1 elements (sign, 2 exponent bits, 1 mantissa bit: magnitudes
 * 0, .5, 1, 1.5, 2, 3, 4, 6).  Blob shapes, the 128-padding of the quantized
 * axis and the row/col option triplets follow the page
 * "primus_turbo_mxfp4_local.py" (ROCm docs download of Primus): its fake
 * (shape-only) dual-quantize op and the arguments of its dual-quantize and
 * FP4 GEMM calls.
 *
 * Conventions shared by every entry point:
 *  - All tensors live in device memory the caller owns; the library allocates
 *    nothing and keeps no state between calls.
 *  - Work is enqueued on `stream` (NULL = the null stream) and runs
 *    asynchronously.  Returned status reflects argument validation and
 *    the launch only; kernels never report errors after launch.
 *  - Validation happens before any launch.  Nothing is written on error, and
 *    there is no fallback path: an unsupported request is an error.
 *  - Sizes are element counts (int64_t); strides are in elements.
 *  - bf16 input x is M x N row-major with row stride ldx >= N elements.
 *  - Thread-safe: calls on different streams may overlap.  Calls that write
 *    the same output buffers race, as with any kernel.
 *
 * Error behaviour: every function returns an mx_status.  mx_last_error()
 * gives a human-readable detail string for the calling thread's last failed
 * call.
 */
#ifndef MXFP4_H
#define MXFP4_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>   /* hipStream_t */

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mx_status {
    MX_SUCCESS = 0,
    MX_ERR_INVALID_ARGUMENT = 1,   /* null pointer, negative size, stride < row length */
    MX_ERR_MISALIGNED = 2,         /* pointer not 16-byte aligned, ldx or ldc not a multiple of 8 */
    MX_ERR_UNSUPPORTED = 3,        /* option combination not implemented (e.g. transposes) */
    MX_ERR_DEVICE_UNSUPPORTED = 4, /* current device is not gfx950 */
    MX_ERR_HIP = 5                 /* HIP runtime error; detail in mx_last_error() */
} mx_status;

/*
 * Blob layouts.
 *
 * MX_LAYOUT_CANONICAL -- the interchange layout of the fake dual-quantize op
 * on the page "primus_turbo_mxfp4_local.py".  For a blob of R rows quantized
 * along an axis of length L, L_pad = cdiv(L,128)*128:
 *   data:  R x L_pad/2 bytes, row-major; element k of a row in byte k/2,
 *          low nibble for even k, high nibble for odd k.
 *   scale: R x L_pad/32 bytes, row-major; byte b scales elements [32b, 32b+32).
 *   Row-wise blob of x: R = M, L = N.  Column-wise blob: R = N, L = M (the
 *   transpose of x, quantized along M).  Padding elements are +0 (nibble 0);
 *   pad-only blocks have scale byte 0.
 *
 * MX_LAYOUT_TILED -- this library's MFMA-native layout, written directly by
 * the quantizers and read by the GEMM with one 16-byte load per lane.
 * Rows are padded to R16 = cdiv(R,16)*16 (pad rows are zero bytes).
 *   data: 1024-byte atoms.  Atom (g, c) holds rows [16g, 16g+16) x k in
 *         [128c, 128c+128) and sits at byte (g * (L_pad/128) + c) * 1024.
 *         Inside an atom, lane = (r%16) + 16*((k%128)/32) owns bytes
 *         [16*lane, 16*lane+16); element k is in byte (k%32)/2 of that slice,
 *         low nibble for even k.  (Lane L holds the 32 elements of row L%16,
 *         k-block L/16: exactly the A/B operand of one 16x16x128 scaled MFMA.)
 *         Total R16 * L_pad/2 bytes.
 *   scale: 256-byte atoms.  Atom (g, h) holds the scales of rows [16g, 16g+16)
 *         and k-blocks [16h, 16h+16) and sits at byte
 *         (g * cdiv(L_pad,512) + h) * 256.  The scale of k-block kb of row r
 *         is byte 4*lane + (kb%16)/4 with lane = (r%16) + 16*(kb%4): each
 *         lane's dword packs its scales for 4 consecutive 128-wide k steps.
 *         Bytes beyond L_pad/32 blocks are 0.  Total R16 * cdiv(L_pad,512) * 16 bytes.
 */
typedef enum mx_layout {
    MX_LAYOUT_CANONICAL = 0,
    MX_LAYOUT_TILED = 1
} mx_layout;

typedef enum mx_dtype {
    MX_BF16 = 0,   /* bfloat16, round to nearest even */
    MX_F32 = 1     /* float32 (verification output of the GEMM) */
} mx_dtype;

/*
 * Per-direction quantization options; the row/col pairs mirror the flag
 * triplets of the dual-quantize op on the page "primus_turbo_mxfp4_local.py"
 * (2D block, stochastic rounding; its Hadamard and shuffle flags have no
 * counterpart here).
 *
 * use_2d_block: 0 = 32-element blocks along the quantized axis; 1 = aligned
 *   32x32 tiles of x share one scale (tile amax), replicated into every
 *   blob row the tile covers; blob shapes are unchanged.
 * use_sr: 0 = round to nearest, ties to even; 1 = stochastic rounding.  The
 *   element with row-major index n = index_base + i*N + j of the logical M x N
 *   tensor draws byte n%16 (little-endian) of Philox-4x32-10 (Salmon et al.,
 *   SC'11) with counter (lo32(n>>4), hi32(n>>4), tensor_id, dir) and key
 *   (lo32(seed), hi32(seed)); dir = 0 for the row-wise blob, 1 for the
 *   column-wise blob.  With neighbouring grid values lo <= v < hi of the scaled
 *   magnitude v, it rounds up iff byte < floor(256*(v-lo)/(hi-lo)).
 * rht: 0 = off; otherwise each 32-element block along the quantized axis is
 *   replaced, before its scale and codes are taken, by the random Hadamard
 *   transform y = c * H32 * D * x evaluated in fp32 (the page
 *   "primus_turbo_mxfp4_local.py" switches "rht" on for the column-wise blobs
 *   of the activation and the gradient, the two wgrad operands, and defines
 *   nothing more; this definition is the library's): D negates position p
 *   when bit p of the first word of Philox-4x32-10 at counter (0, 0, 0, 2),
 *   key (rht, 0) is set; H32 = Sylvester Hadamard matrix, applied as a fast
 *   Walsh-Hadamard transform over position bits 0..4, each (a, b) -> (a + b,
 *   a - b) rounded to fp32; c = fp32(1/sqrt(32)).  Pads count as +0 before
 *   the transform, so pad positions of a block that holds real elements get
 *   codes too.  With use_sr their byte uses the same index formula on padded
 *   coordinates in a counter space of their own: counter word 3 is 2 + dir,
 *   so no pad shares a byte with a real element (and, for the row-wise blob
 *   with N >= 64 and for the column-wise blob, with another pad).  Both
 *   operands of a GEMM must be transformed with the same
 *   rht value along the shared K axis: (H D)^T (H D) c^2 ~= I leaves the
 *   product unchanged.  Not combined with use_2d_block (MX_ERR_UNSUPPORTED).
 * The scale never depends on use_sr.  NULL options = all zero.
 */
typedef struct mx_quant_opts {
    uint32_t use_2d_block;
    uint32_t use_sr;
    uint64_t seed;
    uint32_t tensor_id;
    uint64_t index_base;   /* global element-index offset of x (shards, chunks) */
    uint32_t rht;          /* random Hadamard transform seed, 0 = off */
} mx_quant_opts;

/*
 * Byte sizes of one blob (rows blob rows, quantized along `length`) in
 * `layout`.  Either output pointer may be NULL.  Canonical sizes equal the
 * fake dual-quantize op's shapes: rows * L_pad/2 and rows * L_pad/32.
 * Errors: MX_ERR_INVALID_ARGUMENT (negative size), MX_ERR_UNSUPPORTED (layout).
 */
mx_status mx_blob_bytes(int64_t rows, int64_t length, mx_layout layout,
                        size_t *data_bytes, size_t *scale_bytes);

/*
 * Row-wise MXFP4 quantization of x (M x N bf16, stride ldx): blocks of 32
 * along N, the row-only packer a forward pass with no backward behind it needs
 * (page "Primus PR 1107", the commit that packs rows only when no backward will
 * read the columns; the caller decides, the library never infers grad mode).
 * Outputs: q (data) and s (scales) of the row-wise blob (R = M, L = N) in
 * `layout`, sized by mx_blob_bytes.  Every output byte is written, padding
 * included.  M == 0 or N == 0 is a no-op.
 * Requires x and the outputs 16-byte aligned and ldx % 8 == 0.
 * Errors: INVALID_ARGUMENT, MISALIGNED, UNSUPPORTED, DEVICE_UNSUPPORTED, HIP.
 */
mx_status mx_quantize_rowwise(const void *x, int64_t M, int64_t N, int64_t ldx,
                              const mx_quant_opts *opts, mx_layout layout,
                              void *q, void *s, hipStream_t stream);

/*
 * Dual quantization: the row-wise blob (R = M, L = N) and the column-wise blob
 * (R = N, L = M: x transposed, blocks of 32 along M) from one read of x, as the
 * dual-quantize op on the page "primus_turbo_mxfp4_local.py" returns them
 * (row data, row scale, col data, col scale).  Options are per direction.
 * Same requirements and errors as mx_quantize_rowwise.
 */
mx_status mx_quantize_dual(const void *x, int64_t M, int64_t N, int64_t ldx,
                           const mx_quant_opts *row_opts, const mx_quant_opts *col_opts,
                           mx_layout layout, void *q_row, void *s_row,
                           void *q_col, void *s_col, hipStream_t stream);

/*
 * Quantizer with a multiply prologue: quantizes y = bf16(x * g) (elementwise,
 * each product formed in fp32 and rounded to bf16 nearest-even) exactly as
 * mx_quantize_dual / mx_quantize_rowwise would quantize a stored y, but y is
 * formed in the staging read and never written to memory.  It fuses the
 * last elementwise step of a producer's backward into the packer, the
 * pattern of the page "Primus PR 1107" (its QKV packer computes the
 * gradient during its staging read instead of reading it back from HBM);
 * that page's norm+RoPE backward itself is not part of this library, g
 * carries any elementwise factor (an activation derivative, a mask, a gate).
 * x: M x N bf16, stride ldx; g: M x N bf16, stride ldg.  q_col = s_col =
 * NULL: row-wise blob only.  Options as mx_quantize_dual except rht
 * (MX_ERR_UNSUPPORTED).  Same alignment rules for g as for x.
 * Errors: INVALID_ARGUMENT, MISALIGNED, UNSUPPORTED, DEVICE_UNSUPPORTED, HIP.
 */
mx_status mx_quantize_dual_mul(const void *x, const void *g, int64_t M, int64_t N, int64_t ldx, int64_t ldg,
                               const mx_quant_opts *row_opts, const mx_quant_opts *col_opts,
                               mx_layout layout, void *q_row, void *s_row,
                               void *q_col, void *s_col, hipStream_t stream);

/*
 * Block-scaled FP4 x FP4 GEMM with fp32 accumulation:
 *   C[i][j] = sum_k A[i][k] * B[j][k]   (i < M, j < N, k over the padded K)
 * where A (M rows) and B (N rows) are blobs quantized along K and each
 * element is e2m1(code) * 2^(scale-127).  This is the NT call that the
 * forward (X_row . W_row^T), dgrad (dY_row . W_col^T) and wgrad
 * (dY_col . X_col^T) of the MXFP4 linear on the page
 * "primus_turbo_mxfp4_local.py" all make.
 * transA must be 0 and transB must be 1 (both operands K-contiguous); any
 * other combination returns MX_ERR_UNSUPPORTED.  layout must be
 * MX_LAYOUT_TILED.  K is the logical K; the blobs carry cdiv(K,128)*128.
 * C is M x N row-major with stride ldc >= N, out_dtype MX_BF16 (round to
 * nearest even; overflow to +-Inf) or MX_F32.  A NaN scale byte yields NaN in
 * the affected outputs (hardware-defined propagation).  M == 0 or N == 0 is a
 * no-op; K == 0 writes zeros.
 * Requires 16-byte aligned pointers and ldc % 8 == 0.  Each operand's tiled
 * data blob (cdiv(rows,16)*16 * K_pad/2 bytes) must stay below 2 GiB: the
 * kernels address it with 32-bit buffer offsets (MX_ERR_UNSUPPORTED
 * otherwise, before anything is launched; split the product instead).
 */
mx_status mx_gemm_a4w4(int transA, int transB, int64_t M, int64_t N, int64_t K,
                       const void *A, const void *A_scale,
                       const void *B, const void *B_scale,
                       mx_layout layout, mx_dtype out_dtype,
                       void *C, int64_t ldc, hipStream_t stream);

/*
 * mx_gemm_a4w4 with the linear layer's bias added in the epilogue:
 *   C[i][j] = round(sum_k A[i][k] * B[j][k] + bias[j])
 * bias: N bf16 values (device pointer, 16-byte aligned, caller-owned), added
 * to the fp32 accumulator before the one rounding to out_dtype.  This fuses
 * the separate `output + bias` that the parallel linear layers on the page
 * "primus_turbo_mxfp4_local.py" apply after the FP4 GEMM (there the sum is
 * rounded to bf16 twice; here once).  K == 0 writes bias broadcast over the
 * rows.  Arguments and errors otherwise as mx_gemm_a4w4 (NULL bias:
 * MX_ERR_INVALID_ARGUMENT; misaligned bias: MX_ERR_MISALIGNED).
 */
mx_status mx_gemm_a4w4_bias(int transA, int transB, int64_t M, int64_t N, int64_t K,
                            const void *A, const void *A_scale,
                            const void *B, const void *B_scale,
                            mx_layout layout, mx_dtype out_dtype, const void *bias,
                            void *C, int64_t ldc, hipStream_t stream);

/*
 * ---- Hybrid backward: tensorwise FP8 (E5M2) ----
 * The page "primus_turbo_mxfp4_local.py" offers a backward that re-quantizes
 * the saved bf16 activation, weight and gradient to FP8 E5M2 with one scale
 * per tensor and runs FP8 GEMMs that multiply by both inverse scales.  E5M2
 * per the OCP 8-bit floating point spec (bias 15, 2 mantissa bits, largest
 * finite 57344).  The scale rule is the library's reading (the quantizer's
 * code is not on the pages):
 *   amax = max |x|;  scale = 57344 / amax as an fp32 division (1 if amax is 0
 *   or not finite);  code = E5M2 of the fp32 product x * scale, round to
 *   nearest even, finite overflow saturating to 57344, Inf kept, NaN -> 0x7F
 *   with its sign;  scale_inv = 1 / scale (fp32).
 * FP8 blobs: rows x L_pad bytes (L_pad = cdiv(length,128)*128, pads code 0).
 *   MX_LAYOUT_CANONICAL: row-major.  MX_LAYOUT_TILED: rows padded to 16;
 *   atom (row group g, k-step s of 64) = 1 KB at (g * L_pad/64 + s) * 1024;
 *   lane = (r%16) + 16*((k%64)/16) owns bytes [16 lane, 16 lane + 16),
 *   element k at byte k%16.
 */

/* Bytes of one FP8 blob.  Errors: MX_ERR_INVALID_ARGUMENT, MX_ERR_UNSUPPORTED. */
mx_status mx_fp8_blob_bytes(int64_t rows, int64_t length, mx_layout layout, size_t *bytes);

/*
 * Tensorwise E5M2 quantization of x (M x N bf16, row stride ldx).  q_row
 * (M rows along N) and q_col (N rows along M, the transpose) may each be NULL
 * (not both).  info: device float[2], caller-owned: receives amax in [0] and
 * scale_inv in [1]; [0] is also the reduction's working word, so calls that
 * share an info buffer must not overlap.  Three launches on `stream`.
 * Errors: MX_ERR_INVALID_ARGUMENT (NULL x/info, both outputs NULL, negative
 * sizes, ldx < N), MX_ERR_MISALIGNED (x, outputs or info not 16-byte
 * aligned, ldx % 8), MX_ERR_UNSUPPORTED (layout), MX_ERR_DEVICE_UNSUPPORTED,
 * MX_ERR_HIP.  M == 0 or N == 0 is a no-op.
 */
mx_status mx_quantize_fp8_tw(const void *x, int64_t M, int64_t N, int64_t ldx, mx_layout layout,
                             void *q_row, void *q_col, float *info, hipStream_t stream);

/*
 * C = (A . B^T) * a_scale_inv[0] * b_scale_inv[0] on tensorwise E5M2 blobs
 * (MX_LAYOUT_TILED, both K-contiguous: the NT form of the hybrid backward's
 * dgrad dY_row . W_col^T and wgrad dY_col . X_col^T), fp32 accumulation,
 * bf16 (RNE) or fp32 output.  a_scale_inv / b_scale_inv: device pointers to
 * the inverse scales (the [1] entries of the quantizer's info), read by the
 * kernel, so no host synchronization.  Arguments and errors otherwise as
 * mx_gemm_a4w4 (each FP8 operand blob, cdiv(rows,16)*16 * K_pad bytes, must
 * stay below 2 GiB).
 */
mx_status mx_gemm_f8_tw(int transA, int transB, int64_t M, int64_t N, int64_t K,
                        const void *A, const float *a_scale_inv,
                        const void *B, const float *b_scale_inv,
                        mx_layout layout, mx_dtype out_dtype,
                        void *C, int64_t ldc, hipStream_t stream);

/*
 * ---- FP8 with a scale for each block of 128 ----
 * Blocks of 128 consecutive elements along the quantized axis share one E8M0
 * scale byte c (2^(c-127); use_2d_block: aligned 128 x 128 tiles of x share
 * one, replicated into every blob row that the tile covers) and hold OCP FP8
 * codes.  MAX = 448 (E4M3) or 57344 (E5M2):
 *   c = the smallest byte with max |x| <= MAX * 2^(c-127), so nothing
 *   saturates; 0xFF and zero codes for a block that holds Inf or NaN;
 *   code = x * 2^(127-c) rounded to nearest even.
 * Powers of two, so that the matrix instruction applies the scales itself.
 * Blobs (R rows, quantized axis L, L_pad = cdiv(L,128)*128; pads: code 0,
 * unused scale slots and pad rows: 0):
 *   data as the FP8 blobs above, in either layout (mx_fp8_blob_bytes);
 *   scales, canonical: R x L_pad/128 bytes, row-major;
 *   scales, tiled: 64-byte atoms; atom (g, h) holds rows [16g, 16g+16) and
 *     blocks [4h, 4h+4) and sits at byte (g * cdiv(L_pad,512) + h) * 64; the
 *     byte of row r, block b is 4*(r%16) + b%4 of its atom.
 */
typedef enum mx_fp8_format {
    MX_FP8_E4M3 = 0,
    MX_FP8_E5M2 = 1
} mx_fp8_format;

/* Byte sizes of one blob (either output may be NULL).
 * Errors: MX_ERR_INVALID_ARGUMENT (negative size), MX_ERR_UNSUPPORTED (layout,
 * a size of 2^40 or a blob of 2^62 bytes and above). */
mx_status mx_f8_b128_blob_bytes(int64_t rows, int64_t length, mx_layout layout, size_t *data_bytes,
                                size_t *scale_bytes);

/*
 * Quantization of x (M x N bf16, stride ldx) to the row-wise blob (R = M,
 * L = N) in row_fmt and the column-wise blob (R = N, L = M: x transposed) in
 * col_fmt, from one read of x.  Either pair of outputs may be NULL (not both);
 * its format and options are then ignored.  Options (NULL = all zero):
 * use_2d_block; use_sr and rht must be 0 (MX_ERR_UNSUPPORTED).  Every output
 * byte is written, padding included.  M == 0 or N == 0 is a no-op.
 * Requires x and the outputs 16-byte aligned and ldx % 8 == 0.
 * Errors: INVALID_ARGUMENT, MISALIGNED, UNSUPPORTED (format, layout, options,
 * 2^23 or more 128 x 128 tiles), DEVICE_UNSUPPORTED, HIP.
 */
mx_status mx_quantize_fp8_b128(const void *x, int64_t M, int64_t N, int64_t ldx,
                               int row_fmt, const mx_quant_opts *row_opts,
                               int col_fmt, const mx_quant_opts *col_opts,
                               mx_layout layout, void *q_row, void *s_row,
                               void *q_col, void *s_col, hipStream_t stream);

/*
 * C[i][j] = sum_k A[i][k] * B[j][k] (+ bias[j]) on such blobs (MX_LAYOUT_TILED,
 * both K-contiguous: forward X_row . W_row^T, dgrad dY_row . W_col^T, wgrad
 * dY_col . X_col^T), element = fp8(code) * 2^(scale-127), fp32 accumulation,
 * bf16 (nearest even) or fp32 output.  fmt_a, fmt_b: the operands' formats, any
 * pair.  bias: NULL, or N bf16 values (16-byte aligned), added before the one
 * rounding; the bytes of its last 16-byte block past N are read, never used.
 * K == 0 writes the bias, or zeros.  M == 0 or N == 0 is a no-op.
 * The matrix instruction truncates each product to a multiple of 2^-13 of the
 * largest in its group of 8 along k before it adds in fp32.
 * Arguments, requirements and errors otherwise as mx_gemm_a4w4 (each operand's
 * tiled data blob, cdiv(rows,16)*16 * K_pad bytes, must stay below 2 GiB;
 * MX_ERR_UNSUPPORTED also for 2^23 or more 128 x 128 tiles of C).
 */
mx_status mx_gemm_f8_b128(int transA, int transB, int64_t M, int64_t N, int64_t K,
                          int fmt_a, const void *A, const void *A_scale,
                          int fmt_b, const void *B, const void *B_scale,
                          mx_layout layout, mx_dtype out_dtype, const void *bias,
                          void *C, int64_t ldc, hipStream_t stream);

/*
 * A linear layer's forward pass in one call, y = x . W^T (+ bias): x (M x K
 * bf16, stride ldx) is quantized row-wise to fmt_x and multiplied with the
 * resident blob W (N rows along K, fmt_w); the result is that of
 * mx_quantize_fp8_b128 and mx_gemm_f8_b128 but for the order of the fp32 sums.
 * A few rows (decoding) take one launch.
 * workspace: mx_linear_f8_b128_bytes(M, K) bytes of device memory (NULL if 0),
 * 16-byte aligned; calls that share one must not overlap.
 * Requirements and errors as the two calls (K == 0: x and W may be NULL).
 */
mx_status mx_linear_f8_b128_bytes(int64_t M, int64_t K, size_t *bytes);
mx_status mx_linear_f8_b128(int64_t M, int64_t N, int64_t K, int fmt_x, const void *x, int64_t ldx,
                            int fmt_w, const void *W, const void *W_scale,
                            mx_layout layout, mx_dtype out_dtype, const void *bias,
                            void *y, int64_t ldy, void *workspace, hipStream_t stream);

/*
 * ---- Layers of experts: rows grouped by expert ----
 * A routed linear layer keeps one weight per expert and multiplies each row
 * with the weight of the expert it was routed to, the rows sorted by expert.
 * The groups are given by `group_ends`: device int32[groups], the cumulative
 * end positions; group e is rows [group_ends[e-1], group_ends[e]) of the M
 * grouped rows (from 0 for e = 0), possibly none.  The ends are read by the
 * kernels, never by the host, so a router's output needs no synchronization
 * and a captured graph may be replayed with other ends.  Values are clamped
 * to [0, M], a value below its predecessor counts as the predecessor.  Rows
 * behind the last group belong to none.
 *
 * Grouped blobs (MX_LAYOUT_TILED): the parts of the groups one behind the
 * other, each exactly the tiled blob that mx_quantize_dual gives for the
 * group's n_e rows alone:
 *   row-wise:    rows n_e, length N; group e starts after sum_{j<e}
 *                cdiv(n_j,16)*16 blob rows;
 *   column-wise: rows N, length n_e; its data starts after sum_{j<e}
 *                cdiv(n_j,128) atoms of each of the cdiv(N,16) row groups, its
 *                scales after sum_{j<e} cdiv(n_j,512) scale atoms of each.
 * Bytes behind the last group's part are not written.
 * The weights of the experts (groups of equally many rows, E x N x K as one
 * (E*N) x K tensor with ends N, 2N, ...) are quantized the same way: the
 * row-wise blob is the forward product's B, the column-wise one dgrad's.
 */

/*
 * Bytes that the grouped blobs of M rows of N elements need at most, whatever
 * the ends are.  Each output pointer may be NULL.
 * Errors: MX_ERR_INVALID_ARGUMENT (negative size, groups < 1).
 */
mx_status mx_grouped_blob_bytes(int64_t M, int64_t N, int groups, size_t *row_data_bytes, size_t *row_scale_bytes,
                                size_t *col_data_bytes, size_t *col_scale_bytes);

/*
 * Grouped MXFP4 quantization: the row-wise grouped blob and, when q_col /
 * s_col are given, the column-wise one from the same read of x (q_col = s_col
 * = NULL: row-wise only, as serving needs).
 *   row_index: NULL: grouped row r is row r of x (x_rows must be >= M).
 *     Otherwise device int32[M]: grouped row r is row row_index[r] of x (the
 *     rows of a token routed to several experts are gathered in the same
 *     read); an index outside [0, x_rows) gives a row of zeros.
 *   x: x_rows x N bf16, stride ldx.  Options as mx_quantize_dual (NULL = all
 *     zero); the element index of stochastic rounding is index_base + r*N + j
 *     with the grouped row r.
 *   layout: MX_LAYOUT_TILED.
 * Rows in no group are not read.  M == 0 or N == 0 is a no-op.
 * Requires x and the outputs 16-byte aligned, ldx % 8 == 0, group_ends and
 * row_index 4-byte aligned, and M < 2^30.
 * Errors: INVALID_ARGUMENT, MISALIGNED, UNSUPPORTED (layout, options, M),
 * DEVICE_UNSUPPORTED, HIP.
 */
mx_status mx_quantize_grouped(const void *x, int64_t x_rows, int64_t N, int64_t ldx, const int32_t *row_index,
                              int64_t M, const int32_t *group_ends, int groups, const mx_quant_opts *row_opts,
                              const mx_quant_opts *col_opts, mx_layout layout, void *q_row, void *s_row,
                              void *q_col, void *s_col, hipStream_t stream);

/*
 * Grouped product, forward and dgrad of a layer of experts:
 *   C[r][j] = sum_k A[r][k] * B_e[j][k] (+ bias[e][j])   for the rows r of group e
 * A: a row-wise grouped blob of M rows along K.  B: `groups` tiled blobs of N
 * rows along K, one behind the other (the row-wise grouped blob of weights
 * for forward, the column-wise one for dgrad).  C: M x N, stride ldc, in the
 * grouped order; rows in no group are written as 0.  bias: NULL, or groups x
 * N bf16 values (2-byte aligned), added before the one rounding to out_dtype.
 * The matrix instruction, its accumulation and rounding as mx_gemm_a4w4;
 * K == 0 writes the bias, or zeros.  M == 0 or N == 0 is a no-op.
 * Requires 16-byte aligned operands and C, ldc % 8 == 0.  M rows of A and one
 * group of B must each stay below 2 GiB of blob data.
 * Errors: INVALID_ARGUMENT, MISALIGNED, UNSUPPORTED (layout, out_dtype, sizes),
 * DEVICE_UNSUPPORTED, HIP.
 */
mx_status mx_gemm_a4w4_grouped(int64_t M, int64_t N, int64_t K, const int32_t *group_ends, int groups,
                               const void *A, const void *A_scale, const void *B, const void *B_scale,
                               mx_layout layout, mx_dtype out_dtype, const void *bias, void *C, int64_t ldc,
                               hipStream_t stream);

/*
 * Grouped wgrad of a layer of experts: for each group e
 *   C_e[i][j] = sum_r A[i][r] * B[j][r]   over the group's rows r  (i < N, j < K)
 * A: the column-wise grouped blob of the output gradient (M rows of N), B:
 * the column-wise grouped blob of the input (M rows of K), both with the same
 * ends.  C_e: N x K with row stride ldc at C + e * group_stride elements; a
 * group without rows is written as 0.
 * Requires 16-byte aligned operands and C, ldc % 8 == 0, group_stride % 8 == 0
 * and group_stride >= N * ldc unless groups == 1.  Each blob must stay below
 * 2 GiB of data.
 * Errors as mx_gemm_a4w4_grouped.  N == 0 or K == 0 is a no-op.
 */
mx_status mx_gemm_a4w4_grouped_wgrad(int64_t M, int64_t N, int64_t K, const int32_t *group_ends, int groups,
                                     const void *A, const void *A_scale, const void *B, const void *B_scale,
                                     mx_layout layout, mx_dtype out_dtype, void *C, int64_t ldc,
                                     int64_t group_stride, hipStream_t stream);

/*
 * A whole layer of gated experts for a few tokens (decoding), two launches:
 *   y_t = sum_j w_tj * D_e (silu(G_e x_t) * (U_e x_t)),   e = ids[t][j]
 * with bf16 activations on the experts' MXFP4 weights, fp32 sums; silu(v) =
 * v / (1 + exp(-v)), the product with U_e x_t held as the sum of two bf16 (to 2^-16
 * of it) before D_e.
 *   x: tokens x K bf16, stride ldx.  ids: device int32, tokens x topk; an id
 *     outside [0, experts) counts nothing (an expert that lives elsewhere), one
 *     that a token names more than once counts with the sum of its weights.
 *     weights: device fp32, tokens x topk.
 *   W1: `experts` tiled blobs of 2 * inner rows along K one behind the other, G_e
 *     in rows [0, inner), U_e behind it; W2: `experts` tiled blobs of K rows
 *     along `inner`: the row-wise grouped blobs of mx_quantize_grouped.
 *     Elements that bf16 holds as subnormal numbers may count as 0.
 *   y: tokens x K of out_dtype, stride ldy; every row is written, 0 for a token
 *     without experts.  Inf and NaN of one token reach no other; the order of a
 *     token's fp32 sums goes by how many experts all tokens name together.
 *   workspace: mx_experts_a16w4_bytes bytes, 16-byte aligned; calls that share
 *     one must not overlap.
 * Limits: tokens <= 64, topk <= 32, experts <= 1024, K and inner below 2^24,
 * cdiv(inner,128) * experts below 2^21, x from its first to its last element and one
 * expert's blob below 2 GiB; for more tokens the grouped calls above.  tokens == 0 or
 * K == 0 is a no-op; topk == 0 or inner == 0 writes zeros.
 * Requires x, y, W1, W2, their scales and the workspace 16-byte aligned, ids and
 * weights 4-byte aligned, ldx % 8 == 0 and ldy % 8 == 0.
 * Errors: INVALID_ARGUMENT, MISALIGNED, UNSUPPORTED (layout, out_dtype, sizes),
 * DEVICE_UNSUPPORTED, HIP.
 */
mx_status mx_experts_a16w4_bytes(int64_t tokens, int64_t inner, int topk, size_t *bytes);
mx_status mx_experts_a16w4(int64_t tokens, int64_t K, int64_t inner, int experts, int topk, const void *x,
                           int64_t ldx, const int32_t *ids, const float *weights, const void *W1,
                           const void *W1_scale, const void *W2, const void *W2_scale, mx_layout layout,
                           mx_dtype out_dtype, void *y, int64_t ldy, void *workspace, hipStream_t stream);

/*
 * ---- AdamW over many tensors ----
 * One step of AdamW (Loshchilov and Hutter, decoupled weight decay) for every
 * tensor of a table.  Per element, in fp32 with each operation rounded by
 * itself:
 *   g = grad * grad_scale;  m = beta1*m + (1-beta1)*g;  v = beta2*v + (1-beta2)*(g*g)
 *   param = param*decay - (m / (sqrt(v)*root_factor + eps)) * step_size
 * with decay = 1 - lr*weight_decay, step_size = lr / (1 - beta1^step),
 * root_factor = 1 / sqrt(1 - beta2^step), each rounded once from double.
 *
 * States (MX_STATE_*): fp32, or MXFP8: 32 consecutive elements share an E8M0
 * scale byte c (2^(c-127), 0xFF = NaN block) and each is an OCP E4M3 code; m
 * is held as such, v as its square root.  c is the smallest that keeps the
 * block's largest magnitude within 448: c = max(exponent field of amax - 8 +
 * (mantissa above 1.75), 0).  Codes round to nearest even, or, with use_sr,
 * stochastically: element n draws the word n%4 of Philox-4x32-10 with counter
 * (lo32(n>>2), hi32(n>>2), tensor_id, 4) and key = seed, its low 16 bits for m,
 * its high 16 bits for sqrt(v); with F = the 16 bits that follow the code's
 * bits in the magnitude's binary expansion, it rounds up iff the bits + F
 * carry (unbiased in sqrt(v), so the v it stands for averages above the
 * fp32 state's: in a stationary state by about 0.48 D / sqrt(v), D being the
 * step between codes at sqrt(v), which is 3 to 5% for elements above 2^-14 of
 * their block's largest sqrt(v), and 11, 26 and 75% at 4, 2 and 1 times the
 * smallest code, 2^-16 to 2^-18 of the largest).  A positive sqrt(v) never
 * becomes code 0.  A block that holds Inf or
 * NaN gets scale 0xFF and zero codes.  Zero bytes are the initial states.
 */
typedef enum mx_state_dtype {
    MX_STATE_F32 = 0,
    MX_STATE_MXFP8 = 1
} mx_state_dtype;

/* What changes from step to step. */
typedef struct mx_adamw_step {
    float grad_scale;    /* multiplies the gradient (1 / loss scale, clipping) */
    float decay;
    float step_size;
    float root_factor;
    uint64_t seed;       /* of stochastic rounding: another one each step */
} mx_adamw_step;

typedef struct mx_adamw_tensor {
    void *param;           /* numel of param_dtype, updated in place */
    const void *grad;      /* numel of grad_dtype */
    void *exp_avg;         /* m: numel fp32, or numel E4M3 bytes */
    void *exp_avg_sq;      /* v: numel fp32, or numel E4M3 bytes of sqrt(v) */
    void *exp_avg_scale;   /* MXFP8: cdiv(numel,32) bytes each (any alignment); else NULL */
    void *exp_avg_sq_scale;
    void *param_copy;      /* NULL, or numel bf16: the updated parameter, nearest even */
    int64_t numel;
    uint32_t tensor_id;
} mx_adamw_tensor;

typedef struct mx_adamw_opts {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;          /* counted from 1 */
    double grad_scale;
    uint64_t seed;
    /* MX_F32, or MX_BF16, rounded to nearest even: an update (decay included)
     * below half a bf16 step, 2^-9 to 2^-8 of the parameter, is lost, however
     * often it comes.  Where such updates count: fp32 parameters with a bf16
     * param_copy. */
    int param_dtype;
    int grad_dtype;        /* MX_F32 or MX_BF16 */
    int state_dtype;       /* mx_state_dtype */
    uint32_t use_sr;       /* MXFP8 states: stochastic rounding */
    /* NULL, or a device mx_adamw_step that replaces the values computed from
     * lr, weight_decay, step, grad_scale and seed: a captured graph is replayed
     * with new values in it, and a clipping factor needs no host round trip. */
    const mx_adamw_step *device_step;
} mx_adamw_opts;

/* The step values of opts, as mx_adamw uses them.  Errors: MX_ERR_INVALID_ARGUMENT. */
mx_status mx_adamw_step_values(const mx_adamw_opts *opts, mx_adamw_step *step);

/*
 * One step over tensors[0..count) (a host array, read before the call
 * returns).  Tensors with numel == 0 are skipped; no two tensors may overlap.
 * One launch for up to 48 tensors.
 * Requires param, grad, states and param_copy 16-byte aligned; the bytes of
 * their last 4-byte word past numel are read (never written or used).
 * Errors: MX_ERR_INVALID_ARGUMENT (NULL, count < 0, numel < 0, betas outside
 * [0, 1), eps < 0, step < 1, use_sr not 0 or 1, lr, weight_decay, grad_scale,
 * eps or a step value that is not finite in fp32; values in device_step are
 * used as they are),
 * MX_ERR_MISALIGNED, MX_ERR_UNSUPPORTED (a dtype, numel above 2^33, a bf16
 * copy of bf16 parameters), MX_ERR_DEVICE_UNSUPPORTED, MX_ERR_HIP.
 */
mx_status mx_adamw(const mx_adamw_tensor *tensors, int64_t count, const mx_adamw_opts *opts, hipStream_t stream);

/*
 * ---- The gradients' norm, and clipping ----
 * sum_sq: the sum of the squares of all elements of all tensors, in 64 bits and
 * in a fixed order.  With grad_scale (1 / loss scale):
 *   norm = grad_scale * sqrt(sum_sq)
 *   scale = grad_scale * min(1, max_norm / (norm + 1e-6))
 * scale is mx_adamw's grad_scale: a training step takes it by device_step and
 * the gradients need not be written again, or mx_clip_grads multiplies them.  A
 * norm of Inf gives scale 0 (Inf gradients then become NaN), a NaN one NaN:
 * finite norms are the caller's check.  max_norm = infinity clips nothing:
 * scale is grad_scale, whatever the norm.
 */
typedef struct mx_grad_tensor {
    void *grad;            /* numel of dtype */
    int64_t numel;
    int dtype;             /* MX_F32 or MX_BF16 */
} mx_grad_tensor;

/* In device memory; 8-byte aligned. */
typedef struct mx_grad_norm_info {
    double sum_sq;
    float norm;
    float scale;
} mx_grad_norm_info;

/* Workspace of mx_grad_norm for `count` tensors of any size.
 * Errors: MX_ERR_INVALID_ARGUMENT (count < 0). */
mx_status mx_grad_norm_bytes(int64_t count, size_t *bytes);

/*
 * Norm and scale of tensors[0..count) (a host array, read before the call
 * returns) into info.  step: NULL, or a device mx_adamw_step whose grad_scale
 * becomes the scale (its other fields stay).  max_norm: >= 0, infinity for the
 * norm alone.  Tensors with numel == 0 are skipped; without elements the norm
 * is 0.  workspace: mx_grad_norm_bytes(count) bytes, 8-byte aligned; calls that
 * share it, or info, must not overlap.
 * Requires gradients 16-byte aligned, info and step 8-byte aligned.
 * Errors: MX_ERR_INVALID_ARGUMENT (NULL, count < 0, numel < 0, max_norm < 0 or
 * NaN, grad_scale < 0 or not finite in fp32), MX_ERR_MISALIGNED, MX_ERR_UNSUPPORTED (a dtype,
 * numel above 2^33, count above 2^20), MX_ERR_DEVICE_UNSUPPORTED, MX_ERR_HIP.
 */
mx_status mx_grad_norm(const mx_grad_tensor *tensors, int64_t count, double max_norm, double grad_scale,
                       void *workspace, mx_grad_norm_info *info, mx_adamw_step *step, hipStream_t stream);

/*
 * Norm and scale again from info's sum_sq, for gradients that are spread over
 * processes: mx_grad_norm on each one's part, sum_sq added up over them, then
 * this.  Errors as mx_grad_norm.
 */
mx_status mx_grad_norm_finish(double max_norm, double grad_scale, mx_grad_norm_info *info, mx_adamw_step *step,
                              hipStream_t stream);

/*
 * Every gradient times info's scale, in place: the product in fp32, rounded to
 * nearest even where the gradient is bf16.  No two tensors may overlap.
 * Requirements and errors as mx_grad_norm.
 */
mx_status mx_clip_grads(const mx_grad_tensor *tensors, int64_t count, const mx_grad_norm_info *info,
                        hipStream_t stream);

/* ------------------------------------------------------------------ MXFP6
 *
 * MXFP6: the same 32-element blocks and E8M0 scales with 6-bit elements.
 * The pages name an MXFP6 Flux training campaign (Primus PR 1107) and define
 * none of it; the formats are the OCP MX v1.0 FP6 elements (sec. 5.3.2):
 *   MX_FP6_E2M3: sign, 2 exponent bits (bias 1), 3 mantissa bits; magnitudes
 *     k/8 for k < 8 (subnormal), up to 7.5; emax_elem = 2.
 *   MX_FP6_E3M2: sign, 3 exponent bits (bias 3), 2 mantissa bits; magnitudes
 *     k/16 for k < 4 (subnormal), up to 28; emax_elem = 4.
 * Code = sign << 5 | exponent << mbits | mantissa; no Inf/NaN codes.  Scale
 * byte = max(E(amax) - emax_elem, 0) (0xFF and all-zero codes for a block
 * holding Inf/NaN); elements round to nearest even, or stochastically by the
 * rule of mx_quant_opts, saturating at the largest magnitude.
 *
 * Blob layouts (R rows, quantized axis L, L_pad = cdiv(L,128)*128):
 *   canonical data: R x L_pad*3/4 bytes; element k of a row occupies bits
 *     [6k, 6k+6) of the row read as a little-endian bit string (a 32-element
 *     block is 24 bytes); scales as MX_LAYOUT_CANONICAL.
 *   tiled data: 1536-byte atoms; atom (g, c) = rows [16g, 16g+16) x k in
 *     [128c, 128c+128) at byte (g * (L_pad/128) + c) * 1536.  Lane
 *     (r%16) + 16*((k%128)/32) owns the 24 canonical bytes of its row's
 *     k-block: bytes 0..15 at 16*lane, bytes 16..23 at 1024 + 8*lane (the
 *     six-register operand of the f8f6f4 matrix instruction, split so that
 *     both parts load aligned).  Rows padded to cdiv(R,16)*16 with zeros;
 *     scales exactly as MX_LAYOUT_TILED.
 */
typedef enum mx_fp6_format {
    MX_FP6_E2M3 = 2,
    MX_FP6_E3M2 = 3
} mx_fp6_format;

/* Byte sizes of one MXFP6 blob in `layout` (either output may be NULL).
 * Errors: MX_ERR_INVALID_ARGUMENT (negative size), MX_ERR_UNSUPPORTED (layout). */
mx_status mx_fp6_blob_bytes(int64_t rows, int64_t length, mx_layout layout,
                            size_t *data_bytes, size_t *scale_bytes);

/*
 * MXFP6 quantization of x (M x N bf16, stride ldx): the row-wise blob (R = M,
 * L = N) in row_fmt, and, when q_col / s_col are given, the column-wise blob
 * (R = N, L = M) in col_fmt from the same read of x (q_col = s_col = NULL:
 * row-wise only, as a forward pass with no backward behind it needs).  Options
 * per direction as for mx_quantize_dual, except rht (MX_ERR_UNSUPPORTED).
 * Outputs sized by mx_fp6_blob_bytes; every output byte is written.
 * Requires x and the outputs 16-byte aligned and ldx % 8 == 0.  M == 0 or
 * N == 0 is a no-op.
 * Errors: INVALID_ARGUMENT, MISALIGNED, UNSUPPORTED (format, layout, rht),
 * DEVICE_UNSUPPORTED, HIP.
 */
mx_status mx_quantize_fp6(const void *x, int64_t M, int64_t N, int64_t ldx,
                          int row_fmt, const mx_quant_opts *row_opts,
                          int col_fmt, const mx_quant_opts *col_opts,
                          mx_layout layout, void *q_row, void *s_row,
                          void *q_col, void *s_col, hipStream_t stream);

/*
 * Block-scaled FP6 x FP6 GEMM with fp32 accumulation on tiled MXFP6 blobs:
 *   C[i][j] = sum_k A[i][k] * B[j][k],  element = fp6(code) * 2^(scale-127)
 * with A in fmt_a and B in fmt_b (MX_FP6_E2M3 or MX_FP6_E3M2, mixed allowed).
 * Arguments, layout (MX_LAYOUT_TILED of the MXFP6 blobs), output and errors
 * as mx_gemm_a4w4; MX_ERR_UNSUPPORTED also for an unknown format and when an
 * operand blob (cdiv(rows,16)*16 * K_pad*3/4 bytes) reaches 2 GiB.  The matrix instruction's sum of 64
 * E3M2 x E3M2 products keeps fewer bits than fp32 (measured on MI355X: error
 * up to about 2^-14 of the sum of |products|); E2M3 operands sum exactly.
 */
mx_status mx_gemm_fp6(int transA, int transB, int64_t M, int64_t N, int64_t K,
                      int fmt_a, const void *A, const void *A_scale,
                      int fmt_b, const void *B, const void *B_scale,
                      mx_layout layout, mx_dtype out_dtype,
                      void *C, int64_t ldc, hipStream_t stream);

/*
 * Device-side layout conversion of one blob (rows, length) between the two
 * layouts, asynchronous on `stream`: the tiled layout is the one this
 * library's GEMM reads, the canonical one the interchange shapes of the page
 * "primus_turbo_mxfp4_local.py" (its fake dual-quantize op), so blobs made
 * elsewhere can be fed in and blobs made here handed out.  to_tiled = 1:
 * canonical -> tiled (padding rows and unused scale slots are written as 0);
 * 0: tiled -> canonical.  Device pointers, caller-owned, sized by
 * mx_blob_bytes for their layout; source and destination must not overlap.
 * Errors: MX_ERR_INVALID_ARGUMENT (negative shape, NULL pointer),
 * MX_ERR_MISALIGNED (data or scale pointers not 16-byte aligned),
 * MX_ERR_DEVICE_UNSUPPORTED, MX_ERR_HIP (launch failure).  rows == 0 or
 * length == 0 is a no-op.
 */
mx_status mx_layout_convert(int to_tiled, int64_t rows, int64_t length, const void *q_src,
                            const void *s_src, void *q_dst, void *s_dst, hipStream_t stream);

/*
 * Host-side layout conversion of one blob (rows, length) between the two
 * layouts; plain host pointers, synchronous.  to_tiled = 1: canonical ->
 * tiled; 0: tiled -> canonical.  Destination buffers are sized by
 * mx_blob_bytes for their layout.
 */
mx_status mx_layout_convert_host(int to_tiled, int64_t rows, int64_t length,
                                 const void *q_src, const void *s_src,
                                 void *q_dst, void *s_dst);

/*
 * Device dequantization (a test aid): out[r][k] = element value as float32
 * for r < rows, k < length (logical, unpadded), row stride ldo >= length.
 * Values are exact in float32 for scale bytes <= 252 (the quantizers never
 * emit more for finite input); byte 0xFF gives NaN.
 */
mx_status mx_dequantize(const void *q, const void *s, int64_t rows, int64_t length,
                        mx_layout layout, void *out_f32, int64_t ldo, hipStream_t stream);

/*
 * Measurement aid (not a step of the path): the sustained rate of the
 * block-scaled matrix instruction the GEMMs issue
 * (V_MFMA_SCALE_F32_32X32X64_F8F6F4 with unit scales) for element formats
 * fmt_a x fmt_b (0 E4M3, 1 E5M2, 2 E2M3, 3 E3M2, 4 E2M1: the instruction's own
 * codes), with no memory traffic in its loop, i.e. the ceiling that the
 * chip's clock under matrix work leaves for GEMMs on operands like the given
 * ones (the dense specs assume 2.4 GHz throughout).
 *   operands: device buffer of 64 x 64 uint32 words (16 KB, caller-owned,
 *     16-byte aligned): lane L of every wave uses words [64 L, 64 L + 64) as
 *     4 operand pairs (pair k: A = words 16k..16k+7, B = words 16k+8..16k+15;
 *     an E2M1 operand uses the first 4 words of its 8, an FP6 one the first 6),
 *     one per accumulator chain.
 *   workgroups: >= 1 workgroups of 8 waves (two per SIMD); each wave issues
 *     4 * iters instructions, so one launch performs
 *     workgroups * 8 * 4 * iters * 131072 flops.
 *   out: device float[workgroups * 512] (caller-owned): one sum per lane,
 *     stored so that the work is kept.
 * Asynchronous on `stream`.  Errors: MX_ERR_UNSUPPORTED (format code),
 * MX_ERR_INVALID_ARGUMENT (NULL, workgroups < 1, iters < 1),
 * MX_ERR_MISALIGNED, MX_ERR_DEVICE_UNSUPPORTED, MX_ERR_HIP.
 */
mx_status mx_measure_mfma(int fmt_a, int fmt_b, const void *operands, int workgroups, int64_t iters, float *out,
                          hipStream_t stream);

/*
 * 1 if device `device` is gfx950 (the only target), else 0.  The page
 * "primus_turbo_mxfp4_local.py" has check_mxfp4_support() decide, when a
 * layer is built, whether the FP4 path can run at all, and refuses to build
 * the layer otherwise; this is that check.  Every entry point that launches
 * work repeats it (cached per device) and returns MX_ERR_DEVICE_UNSUPPORTED
 * instead of launching on another device.
 */
int mx_device_supported(int device);

/*
 * Test aid: replaces the device query of every entry point by a fixed
 * architecture name, so that the failure paths can be exercised on any
 * machine.  arch = NULL restores the real query.  With a name other than
 * "gfx950", calls fail with MX_ERR_DEVICE_UNSUPPORTED after validation; with
 * "gfx950" on a machine whose runtime has no usable device, the launch fails
 * and the call returns MX_ERR_HIP with HIP's error text.  The name applies to
 * every device index and to mx_device_supported.  Process-wide; not for use
 * while other threads call the library.  Errors: MX_ERR_INVALID_ARGUMENT (a
 * name of 64 characters or more).
 */
mx_status mx_set_device_arch_override(const char *arch);

/* Static name of a status code. */
const char *mx_status_string(mx_status status);

/* Detail of the calling thread's last failed call ("" if none). */
const char *mx_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
