// A layer of gated experts for a few tokens, in two kernels:
//   y_t = sum_j w_tj down_e(silu(gate_e x_t) * (up_e x_t)),  e = id_tj
// bf16 activations on MXFP4 weights.  With few tokens the weights of the experts
// that are routed to are what has to be read, once each; the activations need
// not be quantized for that: V_CVT_SCALEF32_PK_BF16_FP4 turns two codes and their
// scale into bf16 (exact), and V_MFMA_F32_16X16X32_BF16 multiplies.
//
// The routing is device data.  Each workgroup reads the ids, counts the experts
// that they name in LDS and lists these in order (at most 1024 experts, 64
// tokens); grids go by the most experts that can be named.  An expert's tokens
// are a 64-bit mask: column c of its products is the c-th set bit, so that an
// expert with up to 16 tokens takes one column tile, whichever tokens they are.
//
// Weights go from memory to registers: an atom (16 rows x 128 k, 1 KB) gives lane
// L 32 codes of row L % 16, and the words j of the four lanes of a row are the
// operand of the j-th of four MFMAs, k = 32 (L / 16) + 8 j + 0..7.  The activations
// between the products are written in the order in which the second reads them, a
// column tile of 16 tokens of an expert as 1 KB for each MFMA, each as the sum of
// two bf16.
//
// Sums do not depend on timing: waves split k (up) or the experts' atoms (down)
// and are added in order in LDS; where a row tile of `down` is split over
// workgroups, each writes its sums and the last one to finish adds all in order.
//
// An expert with more than 32 tokens is done in runs of 32, each of which reads its
// weights again.
//
// Bound by latency where the weights are few, else by how many loads are in flight
// (the first kernel: two atoms a wave, three workgroups a CU for their LDS) and by
// the activations, which the second reads from L2 once for every 16 rows of W2, 4
// to 8 KB for each KB of weights.  Measured on MI355X, the two kernels in us, two
// sets of inputs in turn: 1 token, 8 of 64 experts, 2048 x 1024 8.8 + 8.2; 16 tokens,
// 4 of 32, 4096 x 1536 (17 experts named, 114 + 57 MB) 30 + 23, 3.8 and 2.4 TB/s; 64
// tokens, 8 of 64, 2048 x 1024 (48 named, 107 + 53 MB) 38 + 40, 2.8 and 1.3 TB/s.
// With activations of one bf16 the outputs' error grows from 0.0017 to 0.0024 and
// more.

#include <type_traits>

#include "mx_internal.h"

namespace mx {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef float f2_t __attribute__((ext_vector_type(2)));

constexpr int kUpWaves = 4, kDownWaves = 8;
constexpr int kUpTiles = 2;   // atoms of activations in flight per wave, 4 KB a column tile

#define MX_LDS(p) ((__attribute__((address_space(3))) void *)(p))

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
}
constexpr uint32_t kOutOfRange = 0x80000000u;   // past every buffer: loads give 0

__device__ __forceinline__ uint32_t pack(float a, float b) {   // nearest even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2_t{a, b}), bf2_t));
}

// The routing in LDS.
struct Routing {
    uint32_t named[kExpertsMost];  // how often each expert is named
    uint16_t list[kExpertsMost];   // experts that are, in order
    uint16_t tile[kExpertsMost];   // ... and their first column tiles in the workspace
    int count;                     // ... their number
};

// LDS that a launch sizes: the ids, rounded up to 16 bytes, then the kernel's own.
extern __shared__ __attribute__((aligned(1024))) uint8_t s_dynamic[];
__device__ __forceinline__ int *s_ids(int own) { return reinterpret_cast<int *>(s_dynamic + own); }   // tokens x topk

// Reads the ids and lists the experts that they name (ids outside [0, experts)
// name none).  All threads of the workgroup; one wave lists.
__device__ __forceinline__ void read_routing(Routing &r, const ExpertsArgs &a, int *ids, int threads) {
    const int pairs = a.tokens * a.topk, lane = threadIdx.x & 63;
    for (int i = threadIdx.x; i < a.experts; i += threads) r.named[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += threads) {
        const int e = a.ids[i];
        ids[i] = e;
        if ((uint32_t)e < (uint32_t)a.experts) atomicAdd(&r.named[e], 1u);
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        int count = 0, tiles = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 64) {
            const int e = e0 + lane;
            const uint32_t n = e < a.experts ? r.named[e] : 0u;
            const uint64_t is = __builtin_amdgcn_ballot_w64(n > 0);
            int sum = (int)((n + 15) / 16);
            const int mine = sum;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(sum, d, 64);
                if (lane >= d) sum += o;
            }
            if (n > 0) {
                const int at = count + __popcll(is & ((uint64_t(1) << lane) - 1));
                r.list[at] = (uint16_t)e;
                r.tile[at] = (uint16_t)(tiles + sum - mine);
            }
            count += __popcll(is);
            tiles += __builtin_amdgcn_readlane(sum, 63);
        }
        if (lane == 0) r.count = count;
    }
    __syncthreads();
}

// The tokens of expert e as a mask.
__device__ __forceinline__ uint64_t tokens_of(const ExpertsArgs &a, const int *ids, int e, int lane) {
    bool is = false;
    if (lane < a.tokens)
        for (int j = 0; j < a.topk; ++j) is |= ids[lane * a.topk + j] == e;
    return __builtin_amdgcn_ballot_w64(is);
}

// Position of the n-th set bit (n < popcount).
__device__ __forceinline__ int nth_bit(uint64_t mask, int n) {
    int at = 0;
#pragma unroll
    for (int step = 32; step; step >>= 1) {
        const int c = __popcll((mask >> at) & ((uint64_t(1) << step) - 1));
        if (n >= c) {
            n -= c;
            at += step;
        }
    }
    return at;
}

// 32 codes of a lane (4 words) and their scale byte to the weights of MFMA j.
__device__ __forceinline__ float scale_of(uint32_t c) {
    return __uint_as_float(c == 0xFFu ? 0x7FC00000u : c ? c << 23 : 0x00400000u);
}
__device__ __forceinline__ bf8_t weights8(uint32_t w, float scale) {
    const bf2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
    const bf2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    const bf2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
    const bf2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    return bf8_t{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// Where a lane's row lies in a blob of ksteps atoms a row group: byte offsets of
// its codes in atom 0 and of its scale word in scale atom 0.
struct RowAt {
    uint32_t code, scale;
};
__device__ __forceinline__ RowAt row_at(int row, int ksteps, int kgroups, int lane) {
    const uint32_t g = (uint32_t)row >> 4, l = ((uint32_t)row & 15u) + (uint32_t)(lane & 48);
    return {g * (uint32_t)ksteps * 1024u + l * 16u, g * (uint32_t)kgroups * 256u + l * 4u};
}

// Gate and up sums of one wave over the atoms 4 h + wave: MT column tiles.  The
// weights go to registers; an atom's 128 activations of each column, 256
// contiguous bytes of a row of x, to LDS by DMA (4 columns an instruction) and
// back as operands: read from memory in the operands' order, 16 bytes of 16 rows
// at a time, they take 4 times as long as the weights.  16-byte piece p of column
// c lies at p ^ c % 16, so that both sides touch all banks.
template <int RT, int MT, int DEPTH>
__device__ __forceinline__ void up_sum(__amdgpu_buffer_rsrc_t rW, __amdgpu_buffer_rsrc_t rS,
                                       const RowAt (&row)[2][RT], __amdgpu_buffer_rsrc_t rX,
                                       const uint32_t (&x)[MT * 4], int n, uint8_t *lds,
                                       int K, int ksteps, int kgroups, int wave, int lane, v4f (&acc)[2][RT][MT],
                                       int h0 = 0) {
    for (; h0 + DEPTH <= kgroups; h0 += DEPTH) {
        u4_t w[DEPTH][2][RT];
        uint32_t s[DEPTH][2][RT];
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            const int h = h0 + u, c = 4 * h + wave;
            // past K: an offset out of range on its own (the range check subtracts the scalar one from the range)
            const bool in = c < ksteps;
            const int at = in ? c * 1024 : 0;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const uint32_t code = in ? row[t][i].code : kOutOfRange, word = row[t][i].scale;
                    w[u][t][i] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rW, code, at, 0));
                    s[u][t][i] = __builtin_amdgcn_raw_buffer_load_b32(rS, word, h * 256, 0);
                }
        }
        // the operands before are read
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            const int c = 4 * (h0 + u) + wave;
#pragma unroll
            for (int g = 0; g < 4 * MT; ++g)
                if (4 * g < n) {
                    // column 4 g + lane / 16, the piece that belongs at lane % 16
                    const int piece = (lane & 15) ^ ((4 * g + (lane >> 4)) & 15);
                    const uint32_t off = 128 * c + 8 * piece < K ? x[g] + (uint32_t)(256 * c + 16 * piece) : kOutOfRange;
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(rX, MX_LDS(lds + (u * MT * 4 + g) * 1024), 16, off, 0, 0, 0);
                }
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            const int c = 4 * (h0 + u) + wave;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bf8_t b[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int piece = 4 * (lane >> 4) + j;
                    u4_t v = *reinterpret_cast<const u4_t *>(lds + (u * MT + m) * 4096 + (lane & 15) * 256 +
                                                             ((piece ^ (lane & 15)) * 16));
                    if (128 * c + 128 > K) {   // the row's end (wave-uniform): what lies behind it counts 0
                        const int left = K - 128 * c - 8 * piece;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            v[q] &= (2 * q < left ? 0x0000FFFFu : 0u) | (2 * q + 1 < left ? 0xFFFF0000u : 0u);
                    }
                    b[m] = __builtin_bit_cast(bf8_t, v);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const bf8_t a = weights8(w[u][t][i][j], scale_of((s[u][t][i] >> (8 * wave)) & 0xFFu));
#pragma unroll
                        for (int m = 0; m < MT; ++m)
                            acc[t][i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[m], acc[t][i][m], 0, 0, 0);
                    }
            }
        }
    }
    if constexpr (DEPTH > 1)
        up_sum<RT, MT, DEPTH / 2>(rW, rS, row, rX, x, n, lds, K, ksteps, kgroups, wave, lane, acc, h0);
}

// Rows i0 .. i0 + 16 RT - 1 of one expert's activations for its columns [first,
// first + 16 MT), to column tiles `to` on.
template <int RT, int MT>
__device__ __forceinline__ void up_tile(const ExpertsArgs &a, v4f *s_sum, uint8_t *lds, int e, uint64_t mask, int first,
                                        int to, int i0, int wave, int lane) {
    const int ksteps = (int)(padded(a.K) / 128), kgroups = (ksteps + 3) / 4;
    const int n = __popcll(mask) - first, inner = (int)a.inner;
    const int64_t groups = cdiv(2 * a.inner, 16), bytes = groups * ksteps * 1024, sbytes = groups * kgroups * 256;
    const auto rW = make_rsrc(a.W1 + e * bytes, bytes);
    const auto rS = make_rsrc(a.W1s + e * sbytes, sbytes);
    // whole words, which is what the range check goes by
    const auto rX = make_rsrc(a.x, (((int64_t)(a.tokens - 1) * a.ldx + a.K) * 2 + 3) & ~int64_t(3));
    RowAt row[2][RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        // (rows past the inner size: the last one again, not stored)
        const int at = min(i0 + 16 * i + (lane & 15), inner - 1);
        row[0][i] = row_at(at, ksteps, kgroups, lane);
        row[1][i] = row_at(inner + at, ksteps, kgroups, lane);
    }
    uint32_t x[4 * MT];   // byte offsets of the rows of columns 4 g + lane / 16
#pragma unroll
    for (int g = 0; g < 4 * MT; ++g) {
        const int c = 4 * g + (lane >> 4);
        x[g] = c < n ? (uint32_t)(nth_bit(mask, first + c) * a.ldx * 2) : 0u;
    }
    v4f acc[2][RT][MT];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[t][i][m] = v4f{};
    up_sum<RT, MT, kUpTiles / MT>(rW, rS, row, rX, x, n, lds, (int)a.K, ksteps, kgroups, wave, lane, acc);
#pragma unroll
    for (int part = 0; part < RT * MT; ++part) {
        const int t = part / MT, m = part % MT;
        __syncthreads();   // the sums before are read
        s_sum[(2 * wave) * 64 + lane] = acc[0][t][m];
        s_sum[(2 * wave + 1) * 64 + lane] = acc[1][t][m];
        __syncthreads();
        // wave `part` finishes it: lane L holds rows 4 (L / 16) + 0..3 of column L % 16
        if (wave != part || 16 * m + (lane & 15) >= n) continue;
        v4f g = s_sum[lane], u = s_sum[64 + lane];
#pragma unroll
        for (int w = 1; w < kUpWaves; ++w) {
            g += s_sum[(2 * w) * 64 + lane];
            u += s_sum[(2 * w + 1) * 64 + lane];
        }
        const int i = i0 + 16 * t + 4 * (lane >> 4);
        float h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = i + q < inner ? g[q] / (1.0f + expf(-g[q])) * u[q] : 0.0f;
        // For the next product as the sum of two bf16, off by at most 2^-8 of the second, that is 2^-16 of h (one bf16
        // would add an error as large as the output's own rounding).  In the order of its operands: atom i / 128, MFMA
        // i / 8 % 4, lane of the column and of i / 32 % 4; the second bf16 behind the atom's first.
        uint16_t *at = a.h + ((int64_t)(to + m) * (padded(a.inner) / 128) + i / 128) * 4096 + (i / 8 % 4) * 512 +
                       ((lane & 15) + 16 * (i / 32 % 4)) * 8 + i % 8;
        const u2_t hi = {pack(h[0], h[1]), pack(h[2], h[3])};
        float rest[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float r = __uint_as_float(q & 1 ? hi[q >> 1] & 0xFFFF0000u : hi[q >> 1] << 16);
            rest[q] = __builtin_isfinite(r) ? h[q] - r : 0.0f;
        }
        *reinterpret_cast<u2_t *>(at + 2048) = u2_t{pack(rest[0], rest[1]), pack(rest[2], rest[3])};
        *reinterpret_cast<u2_t *>(at) = hi;
    }
}

template <int RT>
__global__ __launch_bounds__(64 * kUpWaves) void experts_up_kernel(ExpertsArgs a, int tiles) {
    __shared__ Routing r;
    v4f *s_sum = reinterpret_cast<v4f *>(s_dynamic);   // once the activations are read
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = blockIdx.x / tiles, tile = blockIdx.x - slot * tiles;
    int *ids = s_ids(kUpWaves * kUpTiles * 4096);
    // the counters of the down kernel
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < kExpertSplits; i += 64 * kUpWaves) a.counters[i] = 0;
    read_routing(r, a, ids, 64 * kUpWaves);
    if (slot >= r.count) return;
    const int e = __builtin_amdgcn_readfirstlane((int)r.list[slot]);
    const int to = __builtin_amdgcn_readfirstlane((int)r.tile[slot]);
    const uint64_t mask = tokens_of(a, ids, e, lane);
    const int n = __popcll(mask);
    uint8_t *lds = s_dynamic + wave * kUpTiles * 4096;
    if (n <= 16) {
        up_tile<RT, 1>(a, s_sum, lds, e, mask, 0, to, 16 * RT * tile, wave, lane);
    } else {
        for (int first = 0; first < n; first += 32) {
            if (first > 0) __syncthreads();   // the sums are read
            up_tile<RT, 2>(a, s_sum, lds, e, mask, first, to + first / 16, 16 * RT * tile, wave, lane);
        }
    }
}

// Sums of a wave over atoms c .. end - 1 of one expert's `down`; h: the lane's
// operands of atom 0, a column tile every `stride` of them.  PARTS: 8, both bf16
// of the activations one after the other, or 4, where columns 8 to 15 hold the
// second ones.
template <int MT, int PARTS, int DEPTH>
__device__ __forceinline__ void down_sum(__amdgpu_buffer_rsrc_t rW, __amdgpu_buffer_rsrc_t rS, RowAt row,
                                         const uint16_t *const (&h)[MT], int c, int end, v4f (&acc)[MT]) {
    for (; c + DEPTH <= end; c += DEPTH) {
        u4_t w[DEPTH], v[DEPTH][MT][PARTS];
        uint32_t s[DEPTH];
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            w[u] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rW, row.code, (c + u) * 1024, 0));
            s[u] = __builtin_amdgcn_raw_buffer_load_b32(rS, row.scale, (c + u) / 4 * 256, 0);
        }
#pragma unroll
        for (int u = 0; u < DEPTH; ++u)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < PARTS; ++j)
                    v[u][m][j] = *reinterpret_cast<const u4_t *>(h[m] + (int64_t)(c + u) * 4096 + j * 512);
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            const float scale = scale_of((s[u] >> (8 * ((c + u) & 3))) & 0xFFu);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf8_t a = weights8(w[u][j], scale);
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int part = 0; part < PARTS; part += 4)
                        acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            a, __builtin_bit_cast(bf8_t, v[u][m][part + j]), acc[m], 0, 0, 0);
            }
        }
    }
    if constexpr (DEPTH > 1) down_sum<MT, PARTS, DEPTH / 2>(rW, rS, row, h, c, end, acc);
}

// Adds an expert's part, for its columns [first, first + 16 MT) in column tiles
// `from` on, to the wave's sums of all tokens, s_sum[token][row].  PAIR: for up to
// 8 columns.
template <int MT, bool PAIR>
__device__ __forceinline__ void down_part(const ExpertsArgs &a, const int *ids, const float *weights, float *s_sum, int e,
                                          uint64_t mask, int first, int from, int n0, int c0, int c1, int lane) {
    const int ksteps = (int)(padded(a.inner) / 128), kgroups = (ksteps + 3) / 4, n = __popcll(mask) - first;
    const int64_t groups = cdiv(a.K, 16), bytes = groups * ksteps * 1024, sbytes = groups * kgroups * 256;
    const uint16_t *h[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        // (columns past the expert's tokens: its last one again, not added)
        const int c = min(lane & (PAIR ? 7 : 15), max(n - 16 * m, 1) - 1);
        h[m] = a.h + (int64_t)(16 * m < n ? from + m : from) * ksteps * 4096 + (c + (lane & 48)) * 8 +
               (PAIR && (lane & 8) ? 2048 : 0);
    }
    v4f acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = v4f{};
    down_sum<MT, PAIR ? 4 : 8, 4 / MT>(make_rsrc(a.W2 + e * bytes, bytes), make_rsrc(a.W2s + e * sbytes, sbytes),
                         row_at(n0 + (lane & 15), ksteps, kgroups, lane), h, c0, c1, acc);
    if constexpr (PAIR)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[0][q] += __shfl_xor(acc[0][q], 8, 64);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int c = 16 * m + (lane & 15);
        if (c >= n) continue;
        const int token = nth_bit(mask, first + c);
        // (an expert that a token names more than once counts with the sum of its weights)
        float weight = 0.0f;
        for (int j = 0; j < a.topk; ++j)
            weight += ids[token * a.topk + j] == e ? weights[token * a.topk + j] : 0.0f;
        v4f *at = reinterpret_cast<v4f *>(s_sum + token * 16 + 4 * (lane >> 4));
        *at += acc[m] * weight;
    }
}

template <bool OUT_BF16>
__device__ __forceinline__ void store_rows(const ExpertsArgs &a, int token, int n, v4f v) {
    const int64_t at = (int64_t)token * a.ldy + n;
    if constexpr (OUT_BF16) {
        uint16_t *dst = static_cast<uint16_t *>(a.y) + at;
        const u2_t w = {pack(v[0], v[1]), pack(v[2], v[3])};
        if (n + 3 < a.K) {
            *reinterpret_cast<u2_t *>(dst) = w;
        } else {
#pragma unroll
            for (int q = 0; q < 3; ++q)
                if (n + q < a.K) dst[q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
        }
    } else {
        float *dst = static_cast<float *>(a.y) + at;
        if (n + 3 < a.K) {
            *reinterpret_cast<v4f *>(dst) = v;
        } else {
#pragma unroll
            for (int q = 0; q < 3; ++q)
                if (n + q < a.K) dst[q] = v[q];
        }
    }
}

// Rows n0 .. n0 + 15 of y for all tokens: part `split` of `splits` of the named
// experts' atoms, the waves taking equal runs of it.
template <bool OUT_BF16>
__global__ __launch_bounds__(64 * kDownWaves) void experts_down_kernel(ExpertsArgs a, int tiles, int splits) {
    __shared__ Routing r;
    __shared__ int s_last;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int split = blockIdx.x / tiles, tile = blockIdx.x - split * tiles, n0 = 16 * tile;
    float *s_sum = reinterpret_cast<float *>(s_dynamic), *own = s_sum + wave * a.tokens * 16;
    int *ids = s_ids(kDownWaves * a.tokens * 64);
    float *weights = reinterpret_cast<float *>(ids + a.tokens * a.topk);
    for (int i = threadIdx.x; i < a.tokens * a.topk; i += 64 * kDownWaves) weights[i] = a.weights[i];
    for (int i = lane; i < a.tokens * 16; i += 64) own[i] = 0.0f;
    read_routing(r, a, ids, 64 * kDownWaves);
    const int per = (int)(padded(a.inner) / 128), total = __builtin_amdgcn_readfirstlane(r.count) * per;
    const int parts = splits * kDownWaves, part = split * kDownWaves + wave;
    int at = (int)((int64_t)total * part / parts);
    const int end = (int)((int64_t)total * (part + 1) / parts);
    while (at < end) {
        const int slot = at / per, c0 = at - slot * per, c1 = min(per, c0 + end - at);
        const int e = __builtin_amdgcn_readfirstlane((int)r.list[slot]);
        const int from = __builtin_amdgcn_readfirstlane((int)r.tile[slot]);
        const uint64_t mask = tokens_of(a, ids, e, lane);
        const int n = __popcll(mask);
        if (n <= 8) {
            down_part<1, true>(a, ids, weights, own, e, mask, 0, from, n0, c0, c1, lane);
        } else if (n <= 16) {
            down_part<1, false>(a, ids, weights, own, e, mask, 0, from, n0, c0, c1, lane);
        } else {
            for (int first = 0; first < n; first += 32)
                down_part<2, false>(a, ids, weights, own, e, mask, first, from + first / 16, n0, c0, c1, lane);
        }
        at += c1 - c0;
    }
    __syncthreads();
    // thread -> token, 4 rows
    static_assert(kExpertTokens * 4 <= 64 * kDownWaves, "a thread for each");
    const int pieces = a.tokens * 4, p = threadIdx.x, n = n0 + 4 * (p & 3);
    const bool live = p < pieces;
    v4f v = {};
    if (live) {
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w) v += *reinterpret_cast<const v4f *>(s_sum + (w * pieces + p) * 4);
    }
    if (splits > 1) {
        // The sums go past the dies' L2s as atomic words of device scope, which are
        // coherent by themselves: once a wave's stores have completed, the counter
        // may follow.  (A device-scope fence writes back the whole L2 instead: 50 us
        // for one token.)
        float *sums = a.sums + (int64_t)tile * splits * pieces * 4;
        if (live)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                __hip_atomic_store(sums + (split * pieces + p) * 4 + e, v[e], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0)
            s_last = __hip_atomic_fetch_add(&a.counters[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == splits - 1;
        __syncthreads();
        if (!s_last || !live) return;
        v = v4f{};
        for (int s = 0; s < splits; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] += __hip_atomic_load(sums + (s * pieces + p) * 4 + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (live && n < a.K) store_rows<OUT_BF16>(a, p >> 2, n, v);
}

}  // namespace

hipError_t launch_experts(const ExpertsArgs &a, mx_dtype out_dtype, hipStream_t stream) {
    const int pairs = a.tokens * a.topk, slots = a.experts < pairs ? a.experts : pairs;
    if (slots > 0) {
        const int rows = expert_row_tiles(slots, a.inner), tiles = (int)(padded(a.inner) / (16 * rows));
        auto kernel = rows == 2 ? experts_up_kernel<2> : experts_up_kernel<1>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(slots * tiles)), dim3(64 * kUpWaves),
                           (unsigned)(kUpWaves * kUpTiles * 4096 + pairs * 4), stream, a, tiles);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int tiles = (int)cdiv(a.K, 16), splits = expert_splits(slots, tiles, a.inner);
    auto kernel = out_dtype == MX_BF16 ? experts_down_kernel<true> : experts_down_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(splits * tiles)), dim3(64 * kDownWaves),
                       (unsigned)(kDownWaves * a.tokens * 64 + pairs * 8), stream, a, tiles, splits);
    return hipGetLastError();
}

}  // namespace mx
