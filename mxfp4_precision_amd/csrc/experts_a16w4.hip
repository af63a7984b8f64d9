// A layer of gated experts for a few tokens, in two kernels:
//   y_t = sum_j w_tj down_e(silu(gate_e x_t) * (up_e x_t)),  e = id_tj
// bf16 activations on MXFP4 weights.  With few tokens the weights of the experts
// that are routed to are what has to be read, once each; the activations need
// not be quantized for that: V_CVT_SCALEF32_PK_BF16_FP4 turns two codes and their
// scale into bf16 (exact), and V_MFMA_F32_16X16X32_BF16 multiplies.
//
// The routing is device data.  Each workgroup reads the ids, marks the experts in
// a bit field in LDS and lists the marked ones in order (at most 1024 experts, 64
// tokens); grids go by the most experts that can be marked.  An expert's tokens
// are a 64-bit mask: column c of its products is the c-th set bit, so that an
// expert with up to 16 tokens takes one column tile, whichever tokens they are.
//
// Weights go from memory to registers: an atom (16 rows x 128 k, 1 KB) gives lane
// L 32 codes of row L % 16, and the words j of the four lanes of a row are the
// operand of the j-th of four MFMAs, k = 32 (L / 16) + 8 j + 0..7; the activations
// are read in that order.
//
// Sums do not depend on timing: waves split k (up) or the experts' atoms (down)
// and are added in order in LDS; where a row tile of `down` is split over
// workgroups, each writes its sums and the last one to finish adds all in order.

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

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
}
constexpr uint32_t kOutOfRange = 0x80000000u;   // past every buffer: loads give 0

__device__ __forceinline__ uint32_t pack(float a, float b) {   // nearest even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2_t{a, b}), bf2_t));
}

// The routing in LDS.
struct Routing {
    uint32_t marks[kExpertsMost / 32];
    uint16_t list[kExpertsMost];   // marked experts in order
    int count;                     // ... their number
};

// LDS that a launch sizes: the ids, rounded up to 16 bytes, then the kernel's own.
extern __shared__ __attribute__((aligned(16))) uint8_t s_dynamic[];
__device__ __forceinline__ int *s_ids() { return reinterpret_cast<int *>(s_dynamic); }   // tokens x topk
__host__ __device__ inline int ids_bytes(const ExpertsArgs &a) { return (a.tokens * a.topk * 4 + 15) & ~15; }

// Reads the ids and lists the marked experts (ids outside [0, experts) mark
// none).  All threads of the workgroup.
__device__ __forceinline__ void read_routing(Routing &r, const ExpertsArgs &a, int threads) {
    const int pairs = a.tokens * a.topk, words = (a.experts + 31) / 32;
    for (int i = threadIdx.x; i < words; i += threads) r.marks[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += threads) {
        const int e = a.ids[i];
        s_ids()[i] = e;
        if ((uint32_t)e < (uint32_t)a.experts) atomicOr(&r.marks[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 32 * words; e += threads) {
        const uint32_t own = r.marks[e >> 5];
        int rank = __popc(own & ((1u << (e & 31)) - 1u));
        for (int w = 0; w < (e >> 5); ++w) rank += __popc(r.marks[w]);
        if ((own >> (e & 31)) & 1u) r.list[rank] = (uint16_t)e;
        if (e == 32 * words - 1) r.count = rank + (int)(own >> 31);
    }
    __syncthreads();
}

// The tokens of expert e as a mask.
__device__ __forceinline__ uint64_t tokens_of(const ExpertsArgs &a, int e, int lane) {
    bool is = false;
    if (lane < a.tokens)
        for (int j = 0; j < a.topk; ++j) is |= s_ids()[lane * a.topk + j] == e;
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

// The first place of expert e among a token's ids.
__device__ __forceinline__ int place_of(const ExpertsArgs &a, int e, int token) {
    int at = 0;
    for (int j = a.topk - 1; j >= 0; --j)
        if (s_ids()[token * a.topk + j] == e) at = j;
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

// 8 activations from p + k of a row of n, 0 past its end.  Rows start at
// 16-byte boundaries and `k` is a multiple of 8.
__device__ __forceinline__ u4_t load8(const uint16_t *p, int64_t k, int64_t n) {
    u4_t v = {};
    if (k >= n) return v;
    if (k + 8 <= n) return *reinterpret_cast<const u4_t *>(p + k);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = p[k + e < n ? k + e : n - 1];
        v[e >> 1] |= (k + e < n ? b : 0u) << (16 * (e & 1));
    }
    return v;
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

// Gate and up sums of one wave over the atoms 4 h + wave: MT column tiles.
template <int MT, int DEPTH>
__device__ __forceinline__ void up_sum(__amdgpu_buffer_rsrc_t rW, __amdgpu_buffer_rsrc_t rS, RowAt gate, RowAt up,
                                       const uint16_t *const (&x)[MT], int64_t K, int ksteps, int kgroups, int wave,
                                       int lane, v4f (&acc)[2][MT], int h0 = 0) {
    for (; h0 + DEPTH <= kgroups; h0 += DEPTH) {
        u4_t w[DEPTH][2], v[DEPTH][MT][4];
        uint32_t s[DEPTH][2];
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            const int h = h0 + u, c = 4 * h + wave;
            // past K: an offset out of range on its own (the range check subtracts the scalar one from the range)
            const bool in = c < ksteps;
            const int at = in ? c * 1024 : 0;
            w[u][0] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rW, in ? gate.code : kOutOfRange, at, 0));
            w[u][1] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rW, in ? up.code : kOutOfRange, at, 0));
            s[u][0] = __builtin_amdgcn_raw_buffer_load_b32(rS, gate.scale, h * 256, 0);
            s[u][1] = __builtin_amdgcn_raw_buffer_load_b32(rS, up.scale, h * 256, 0);
        }
        const int64_t k0 = 128 * (int64_t)(4 * h0 + wave);
        const auto load = [&](auto whole) {
#pragma unroll
            for (int u = 0; u < DEPTH; ++u)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int64_t k = k0 + 512 * u + 32 * (lane >> 4) + 8 * j;
                        if constexpr (decltype(whole)::value) v[u][m][j] = *reinterpret_cast<const u4_t *>(x[m] + k);
                        else v[u][m][j] = load8(x[m], k, K);
                    }
        };
        if (k0 + 512 * (DEPTH - 1) + 128 <= K) load(std::true_type{});   // (wave-uniform)
        else load(std::false_type{});
#pragma unroll
        for (int u = 0; u < DEPTH; ++u)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float scale = scale_of((s[u][t] >> (8 * wave)) & 0xFFu);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf8_t a = weights8(w[u][t][j], scale);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        acc[t][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf8_t, v[u][m][j]),
                                                                            acc[t][m], 0, 0, 0);
                }
            }
    }
    if constexpr (DEPTH > 1)
        up_sum<MT, DEPTH / 2>(rW, rS, gate, up, x, K, ksteps, kgroups, wave, lane, acc, h0);
}

// Rows i0 .. i0 + 15 of one expert's activations for its tokens, MT column tiles.
template <int MT>
__device__ __forceinline__ void up_tile(const ExpertsArgs &a, v4f *s_sum, int e, uint64_t mask,
                                        int i0, int wave, int lane) {
    const int ksteps = (int)(padded(a.K) / 128), kgroups = (ksteps + 3) / 4;
    const int n = __popcll(mask), inner = (int)a.inner;
    const int64_t groups = cdiv(2 * a.inner, 16), bytes = groups * ksteps * 1024, sbytes = groups * kgroups * 256;
    const auto rW = make_rsrc(a.W1 + e * bytes, bytes);
    const auto rS = make_rsrc(a.W1s + e * sbytes, sbytes);
    // (rows past the inner size: the last one again, not stored)
    const int row = min(i0 + (lane & 15), inner - 1);
    const uint16_t *x[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int c = 16 * m + (lane & 15);
        // (columns past the expert's tokens: its first one again, not stored)
        x[m] = a.x + (int64_t)nth_bit(mask, c < n ? c : 0) * a.ldx;
    }
    v4f acc[2][MT];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] = v4f{};
    up_sum<MT, MT == 1 ? 4 : MT == 2 ? 2 : 1>(rW, rS, row_at(row, ksteps, kgroups, lane),
                                              row_at(inner + row, ksteps, kgroups, lane), x, a.K, ksteps, kgroups,
                                              wave, lane, acc);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m > 0) __syncthreads();
        s_sum[(2 * wave) * 64 + lane] = acc[0][m];
        s_sum[(2 * wave + 1) * 64 + lane] = acc[1][m];
        __syncthreads();
        // wave m finishes column tile m: lane L holds rows i0 + 4 (L / 16) + 0..3 of column L % 16
        const int c = 16 * m + (lane & 15);
        if (wave != m || c >= n) continue;
        v4f g = s_sum[lane], u = s_sum[64 + lane];
#pragma unroll
        for (int w = 1; w < kUpWaves; ++w) {
            g += s_sum[(2 * w) * 64 + lane];
            u += s_sum[(2 * w + 1) * 64 + lane];
        }
        const int token = nth_bit(mask, c), pair = token * a.topk + place_of(a, e, token);
        const int i = i0 + 4 * (lane >> 4);
        float h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = i + q < inner ? g[q] / (1.0f + expf(-g[q])) * u[q] : 0.0f;
        // bf16, the type of the next product's operand: off by at most 2^-8 of each, as every activation held in bf16
        *reinterpret_cast<u2_t *>(a.h + (int64_t)pair * padded(a.inner) + i) = u2_t{pack(h[0], h[1]), pack(h[2], h[3])};
    }
}

__global__ __launch_bounds__(64 * kUpWaves) void experts_up_kernel(ExpertsArgs a, int tiles) {
    __shared__ Routing r;
    __shared__ v4f s_sum[kUpWaves * 2 * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = blockIdx.x / tiles, tile = blockIdx.x - slot * tiles;
    // the counters of the down kernel
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < kExpertSplits; i += 64 * kUpWaves) a.counters[i] = 0;
    read_routing(r, a, 64 * kUpWaves);
    if (slot >= r.count) return;
    const int e = __builtin_amdgcn_readfirstlane((int)r.list[slot]);
    const uint64_t mask = tokens_of(a, e, lane);
    const int n = __popcll(mask);
    if (n <= 16) up_tile<1>(a, s_sum, e, mask, 16 * tile, wave, lane);
    else if (n <= 32) up_tile<2>(a, s_sum, e, mask, 16 * tile, wave, lane);
    else up_tile<4>(a, s_sum, e, mask, 16 * tile, wave, lane);
}

// Sums of a wave over atoms c0 .. c0 + n - 1 of one expert's `down`.
template <int MT, int DEPTH>
__device__ __forceinline__ void down_sum(__amdgpu_buffer_rsrc_t rW, __amdgpu_buffer_rsrc_t rS, RowAt row,
                                         const uint16_t *const (&h)[MT], int c, int end, int lane,
                                         v4f (&acc)[MT]) {
    for (; c + DEPTH <= end; c += DEPTH) {
        u4_t w[DEPTH], v[DEPTH][MT][4];
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
                for (int j = 0; j < 4; ++j)
                    v[u][m][j] = *reinterpret_cast<const u4_t *>(h[m] + 128 * (c + u) + 32 * (lane >> 4) + 8 * j);
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            const float scale = scale_of((s[u] >> (8 * ((c + u) & 3))) & 0xFFu);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf8_t a = weights8(w[u][j], scale);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf8_t, v[u][m][j]), acc[m],
                                                                     0, 0, 0);
            }
        }
    }
    if constexpr (DEPTH > 1) down_sum<MT, DEPTH / 2>(rW, rS, row, h, c, end, lane, acc);
}

// Adds an expert's part to the wave's sums of all tokens, s_sum[token][row].
template <int MT>
__device__ __forceinline__ void down_part(const ExpertsArgs &a, float *s_sum, int e, uint64_t mask,
                                          int n0, int c0, int c1, int lane) {
    const int ksteps = (int)(padded(a.inner) / 128), kgroups = (ksteps + 3) / 4, n = __popcll(mask);
    const int64_t groups = cdiv(a.K, 16), bytes = groups * ksteps * 1024, sbytes = groups * kgroups * 256;
    const int64_t wide = padded(a.inner);
    const uint16_t *h[MT];
    float weight[MT];
    int token[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int c = 16 * m + (lane & 15);
        token[m] = nth_bit(mask, c < n ? c : 0);
        h[m] = a.h + ((int64_t)token[m] * a.topk + place_of(a, e, token[m])) * wide;
        weight[m] = 0.0f;
        // (an expert that a token names more than once counts with the sum of its weights)
        for (int j = 0; j < a.topk; ++j)
            if (s_ids()[token[m] * a.topk + j] == e) weight[m] += a.weights[token[m] * a.topk + j];
        if (c >= n) token[m] = -1;   // past the expert's tokens: its first one again, not added
    }
    v4f acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = v4f{};
    down_sum<MT, MT == 1 ? 4 : MT == 2 ? 2 : 1>(make_rsrc(a.W2 + e * bytes, bytes), make_rsrc(a.W2s + e * sbytes, sbytes),
                                                row_at(n0 + (lane & 15), ksteps, kgroups, lane), h, c0, c1, lane,
                                                acc);
#pragma unroll
    for (int m = 0; m < MT; ++m)
        if (token[m] >= 0) {
            v4f *at = reinterpret_cast<v4f *>(s_sum + token[m] * 16 + 4 * (lane >> 4));
            *at += acc[m] * weight[m];
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

// Rows n0 .. n0 + 15 of y for all tokens: part `split` of `splits` of the marked
// experts' atoms, the waves taking equal runs of it.
template <bool OUT_BF16>
__global__ __launch_bounds__(64 * kDownWaves) void experts_down_kernel(ExpertsArgs a, int tiles, int splits) {
    __shared__ Routing r;
    __shared__ int s_last;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int split = blockIdx.x / tiles, tile = blockIdx.x - split * tiles, n0 = 16 * tile;
    float *s_sum = reinterpret_cast<float *>(s_dynamic + ids_bytes(a)), *own = s_sum + wave * a.tokens * 16;
    for (int i = lane; i < a.tokens * 16; i += 64) own[i] = 0.0f;
    read_routing(r, a, 64 * kDownWaves);
    const int per = (int)(padded(a.inner) / 128), total = __builtin_amdgcn_readfirstlane(r.count) * per;
    const int parts = splits * kDownWaves, part = split * kDownWaves + wave;
    int at = (int)((int64_t)total * part / parts);
    const int end = (int)((int64_t)total * (part + 1) / parts);
    while (at < end) {
        const int slot = at / per, c0 = at - slot * per, c1 = min(per, c0 + end - at);
        const int e = __builtin_amdgcn_readfirstlane((int)r.list[slot]);
        const uint64_t mask = tokens_of(a, e, lane);
        const int n = __popcll(mask);
        if (n <= 16) down_part<1>(a, own, e, mask, n0, c0, c1, lane);
        else if (n <= 32) down_part<2>(a, own, e, mask, n0, c0, c1, lane);
        else down_part<4>(a, own, e, mask, n0, c0, c1, lane);
        at += c1 - c0;
    }
    __syncthreads();
    // thread -> token, 4 rows
    const int token = threadIdx.x >> 2, q = threadIdx.x & 3;
    const bool live = token < a.tokens;
    v4f v = {};
    if (live) {
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w) v += *reinterpret_cast<const v4f *>(s_sum + (w * a.tokens + token) * 16 + 4 * q);
    }
    if (splits > 1) {
        // The sums go past the dies' L2s as atomic words of device scope, which are
        // coherent by themselves: once a wave's stores have completed, the counter
        // may follow.  (A device-scope fence writes back the whole L2 instead: 50 us
        // of one token's 13.)
        float *sums = a.sums + (int64_t)tile * splits * a.tokens * 16;
        float *own_sums = sums + (split * a.tokens * 4 + (int)threadIdx.x) * 4;
        if (live)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                __hip_atomic_store(own_sums + e, v[e], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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
                v[e] += __hip_atomic_load(sums + (s * a.tokens * 4 + (int)threadIdx.x) * 4 + e, __ATOMIC_RELAXED,
                                          __HIP_MEMORY_SCOPE_AGENT);
    }
    if (live && n0 + 4 * q < a.K) store_rows<OUT_BF16>(a, token, n0 + 4 * q, v);
}

}  // namespace

hipError_t launch_experts(const ExpertsArgs &a, mx_dtype out_dtype, hipStream_t stream) {
    const int pairs = a.tokens * a.topk, slots = a.experts < pairs ? a.experts : pairs;
    const int up_tiles = (int)(padded(a.inner) / 16), down_tiles = (int)cdiv(a.K, 16);
    if (slots > 0) {
        hipLaunchKernelGGL(experts_up_kernel, dim3((unsigned)(slots * up_tiles)), dim3(64 * kUpWaves),
                           (unsigned)ids_bytes(a), stream, a, up_tiles);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int splits = expert_splits(slots, a.K, a.inner);
    auto kernel = out_dtype == MX_BF16 ? experts_down_kernel<true> : experts_down_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(splits * down_tiles)), dim3(64 * kDownWaves),
                       (unsigned)(ids_bytes(a) + kDownWaves * a.tokens * 64), stream, a, down_tiles, splits);
    return hipGetLastError();
}

}  // namespace mx
