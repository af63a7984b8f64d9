// One AdamW step over many tensors in as few launches as kernel arguments
// hold descriptors.
//
// Per element, in fp32 with every operation rounded by itself (contraction
// off, so that the 8-bit states have one definition to the bit):
//   g = grad * grad_scale
//   m = beta1 m + (1 - beta1) g          v = beta2 v + (1 - beta2) (g g)
//   p = p decay - (m / (sqrt(v) vfac + eps)) step_size
// decay = 1 - lr weight_decay, step_size = lr / (1 - beta1^t), vfac =
// 1 / sqrt(1 - beta2^t), rounded from double on the host.
//
// 8-bit states are MXFP8 blocks: 32 consecutive elements share an E8M0 scale
// byte and are E4M3 (OFP8) codes; what is held of v is sqrt(v), which halves
// its range of exponents.  The scale is the smallest power of two that keeps
// the block's largest value within 448 (the OCP rule, which saturates values
// up to 512, would take up to 12.5% off the largest second moment of a block
// each step).  With beta2 near 1 a step changes sqrt(v) by less than half an
// E4M3 step, so nearest rounding would hold it for ever: stochastic rounding
// (16 bits of Philox-4x32-10 for each state and element) is the mode meant
// for training.  It is unbiased in sqrt(v), so the v it stands for averages
// higher by the held value's variance: for gradients of constant variance
// 0.48 D / sqrt(v) (D: the step between codes), 3.5% at beta2 0.99 and 4.6% at
// 0.999, 26% at twice the smallest code.  A positive sqrt(v) keeps at least the smallest code: at 0
// the next update would be divided by eps.
//
// A lane owns 8 consecutive elements, so a block's largest value is found in
// its 4 lanes with two DPP quad permutes.  Measured on MI355X:
//  - fp32 states, fp32 parameters, bf16 gradients and copy (28 bytes an
//    element), 76M elements: 395 us, 5.4 TB/s; bound by memory (a 4 GiB copy
//    moves 4.8 TB/s).  Plain fp32 loads, as the lines are written again at
//    once: 418 us with non-temporal ones.
//  - MXFP8 states, bf16 parameters and gradients, stochastic (10.1 bytes), 201M
//    elements: 385 us, 5.3 TB/s, memory and arithmetic about even (65 vector
//    instructions an element, 13 of them Philox).  The earlier forms of the
//    decode (ldexp and a NaN select per value), the encode (codes masked and
//    shifted one by one) and the square root took 434 us.

#include <cstddef>
#include <cstring>

#include "mx_internal.h"

namespace mx {
namespace {

typedef float f4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
typedef float f2_t __attribute__((ext_vector_type(2)));

constexpr int kLaneElems = 8;
constexpr int kThreads = 256;
constexpr int kChunk = kThreads * kLaneElems;   // elements of one workgroup pass

__device__ __forceinline__ void philox(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c[0];
        const uint64_t p1 = (uint64_t)0xCD9E8D57u * c[2];
        const uint32_t n0 = __builtin_amdgcn_bitop3_b32((uint32_t)(p1 >> 32), c[1], k0, 0x96);
        const uint32_t n2 = __builtin_amdgcn_bitop3_b32((uint32_t)(p0 >> 32), c[3], k1, 0x96);
        c[0] = n0; c[1] = (uint32_t)p1; c[2] = n2; c[3] = (uint32_t)p0;
        k0 += 0x9E3779B9u; k1 += 0xBB67AE85u;
    }
}

// A workgroup's chunk of an array, as a buffer: n elements of `size` bytes at
// p, rounded up to whole dwords, which is what the range check of a load goes
// by (p is 16-byte aligned, so they lie in the array's last 16-byte block).
// Loads past the end read 0, without the branches that would make a tensor's
// last chunk wait for one array after the other.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_of(const void *p, int64_t first, int n, int size) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(static_cast<const uint8_t *>(p)) + first * size, (short)0,
                                             (n * size + 3) & ~3, 0x00020000);
}
constexpr int kNT = 2;   // cache policy: non-temporal

// Elements i .. i + 7 of a chunk.
template <bool F32>
__device__ __forceinline__ void load8(__amdgpu_buffer_rsrc_t r, int i, float (&v)[8]) {
    if constexpr (F32) {
        const f4_t a = __builtin_bit_cast(f4_t, __builtin_amdgcn_raw_buffer_load_b128(r, i * 4, 0, 0));
        const f4_t b = __builtin_bit_cast(f4_t, __builtin_amdgcn_raw_buffer_load_b128(r, i * 4 + 16, 0, 0));
#pragma unroll
        for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
    } else {
        const u4_t a = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(r, i * 2, 0, kNT));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(a[e] << 16);
            v[2 * e + 1] = __uint_as_float(a[e] & 0xFFFF0000u);
        }
    }
}

// The first `left` of eight elements to p + i; FULL: all eight.
template <bool FULL, bool F32>
__device__ __forceinline__ void store8(void *p, int64_t i, int left, const float (&v)[8]) {
    if constexpr (F32) {
        float *s = static_cast<float *>(p) + i;
        if (FULL || left >= 8) {
            __builtin_nontemporal_store(f4_t{v[0], v[1], v[2], v[3]}, reinterpret_cast<f4_t *>(s));
            __builtin_nontemporal_store(f4_t{v[4], v[5], v[6], v[7]}, reinterpret_cast<f4_t *>(s) + 1);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) s[e] = v[e];
        }
    } else {
        uint32_t w[4];   // nearest even
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2_t{v[2 * e], v[2 * e + 1]}), bf2_t));
        uint16_t *s = static_cast<uint16_t *>(p) + i;
        if (FULL || left >= 8) {
            __builtin_nontemporal_store(u4_t{w[0], w[1], w[2], w[3]}, reinterpret_cast<u4_t *>(s));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) s[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// The values they stand for: E4M3 times 2^(c - 127), NaN for c = 0xFF.  The
// scale is an fp32 number for every c < 0xFF (2^-127 a subnormal one) and the
// product exact.
__device__ __forceinline__ void decode8(u2_t w, uint32_t c, float (&v)[8]) {
    const float scale = c == 0xFFu ? __uint_as_float(0x7FC00000u)
                                   : __builtin_ldexpf(__uint_as_float(0x00400000u), (int)c);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
        const f2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
        v[4 * h] = a[0] * scale; v[4 * h + 1] = a[1] * scale;
        v[4 * h + 2] = b[0] * scale; v[4 * h + 3] = b[1] * scale;
    }
}

// A block's scale byte from its largest magnitude as an fp32 pattern: the
// exponent field less 8, one more when the mantissa is above 1.75 (448 =
// 1.75 2^8), which the carry of the addition gives; 0xFF for Inf or NaN.
__device__ __forceinline__ uint32_t scale_of(uint32_t amax) {
    if (amax >= 0x7F800000u) return 0xFFu;
    const int c = (int)((amax + 0x1FFFFFu) >> 23) - 8;
    return c > 0 ? (uint32_t)c : 0u;
}

__device__ __forceinline__ uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Largest pattern over the 4 lanes of a block.
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
    v = max_u(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
    return max_u(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
}

// Byte 3 of four words.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_amdgcn_perm(b, a, 0x0C0C0703u) | __builtin_amdgcn_perm(d, c, 0x07030C0Cu);
}

// Eight values -> E4M3 codes under scale byte c.  u = |x| 2^(7 - c) as an
// fp32 pattern has E4M3's fields on top (its subnormal step falls on the fp32
// subnormal grid): the code is u >> 20, plus 1 when the 16 bits below it
// exceed what the random bits leave (SR) or by the nearest-even rule.  It is
// formed in the top byte of u << 4, where one permute gathers two codes.
// ROOT: values >= 0; its random bits are the words' upper halves.
template <bool SR, bool ROOT>
__device__ __forceinline__ u2_t encode8(const float (&x)[8], uint32_t c, const uint32_t (&bits)[8]) {
    uint32_t s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t u = __float_as_uint(__builtin_ldexpf(__builtin_fabsf(x[e]), 7 - (int)c));
        uint32_t v;
        if constexpr (SR)   // 16 random bits at bits 8..23
            v = (u << 4) + __builtin_amdgcn_perm(bits[e], bits[e], ROOT ? 0x0C03020Cu : 0x0C01000Cu);
        else
            v = (u + 0x7FFFFu + ((u >> 20) & 1u)) << 4;
        v = v < 0x7EFFFFFFu ? v : 0x7EFFFFFFu;
        if constexpr (ROOT) {   // a positive value keeps at least the smallest code
            const uint32_t least = x[e] > 0.0f ? 1u << 24 : 0u;
            v = v > least ? v : least;
        }
        s[e] = v;
    }
    u2_t w = {top_bytes(s[0], s[1], s[2], s[3]), top_bytes(s[4], s[5], s[6], s[7])};
    if constexpr (!ROOT) {
        const auto bit = [&](int e) { return __float_as_uint(x[e]); };
        w[0] |= top_bytes(bit(0), bit(1), bit(2), bit(3)) & 0x80808080u;
        w[1] |= top_bytes(bit(4), bit(5), bit(6), bit(7)) & 0x80808080u;
    }
    return c == 0xFFu ? u2_t{0u, 0u} : w;
}

template <bool FULL>
__device__ __forceinline__ void store_codes(uint8_t *p, int64_t i, int left, u2_t w) {
    if (FULL || left >= 8) {
        __builtin_nontemporal_store(w, reinterpret_cast<u2_t *>(p + i));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) p[i + e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
    }
}

// Square roots, rounded to nearest.  The compiler's own sequence scales small
// arguments and tests for special ones; where a wave has none of either
// (arguments in [2^-96, 2^96]) v_sqrt_f32, off by at most one step, and the
// residuals of its two neighbours do.
__device__ __forceinline__ void sqrt8(const float (&v)[8], float (&root)[8]) {
#pragma clang fp contract(off)
    uint32_t lo = ~0u, hi = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(v[e]);
        lo = b < lo ? b : lo;
        hi = max_u(hi, b);
    }
    if (__builtin_amdgcn_ballot_w64(lo < 0x0F800000u || hi > 0x6F800000u) == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float s = __builtin_amdgcn_sqrtf(v[e]);
            const float below = __uint_as_float(__float_as_uint(s) - 1u), above = __uint_as_float(__float_as_uint(s) + 1u);
            float r = __builtin_fmaf(-below, s, v[e]) <= 0.0f ? below : s;
            root[e] = __builtin_fmaf(-above, s, v[e]) > 0.0f ? above : r;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) root[e] = __builtin_sqrtf(v[e]);
    }
}

// This lane's eight elements of the chunk from `first` on (n elements; FULL:
// kChunk of them).
template <bool FULL, bool P32, bool G32, bool S8, bool SR, typename TABLE>
__device__ __forceinline__ void update8(const TABLE &b, const AdamwItem &it, const mx_adamw_step &h, int64_t first,
                                        int n) {
#pragma clang fp contract(off)
    const int local = threadIdx.x * kLaneElems, left = FULL ? 8 : (n - local < 0 ? 0 : (n - local > 8 ? 8 : n - local));
    const int64_t i = first + local;
    float p[8], g[8], m[8], v[8];
    load8<G32>(chunk_of(it.grad, first, n, G32 ? 4 : 2), local, g);
    load8<P32>(chunk_of(it.param, first, n, P32 ? 4 : 2), local, p);
    uint32_t bits[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    // the random words while the loads are in flight
    const auto draw = [&]() {
        const uint64_t k = (uint64_t)i >> 2;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t c[4] = {(uint32_t)(k + q), (uint32_t)((k + q) >> 32), it.tensor_id, 4u};
            philox(c, (uint32_t)h.seed, (uint32_t)(h.seed >> 32));
#pragma unroll
            for (int e = 0; e < 4; ++e) bits[4 * q + e] = c[e];
        }
    };
    if constexpr (S8) {
        u2_t wm = __builtin_bit_cast(u2_t, __builtin_amdgcn_raw_buffer_load_b64(chunk_of(it.m, first, n, 1), local, 0, kNT));
        u2_t wv = __builtin_bit_cast(u2_t, __builtin_amdgcn_raw_buffer_load_b64(chunk_of(it.v, first, n, 1), local, 0, kNT));
        uint32_t cm = 0, cv = 0;
        if (FULL || left > 0) {
            cm = it.ms[i / 32];
            cv = it.vs[i / 32];
        }
        if constexpr (SR) draw();
        if constexpr (!FULL) {   // a dword that the end cuts holds other bytes too
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int keep = left - 4 * e;
                const uint32_t mask = keep >= 4 ? ~0u : (keep <= 0 ? 0u : (1u << (8 * keep)) - 1u);
                wm[e] &= mask;
                wv[e] &= mask;
            }
        }
        decode8(wm, cm, m);
        decode8(wv, cv, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * v[e];
    } else {
        load8<true>(chunk_of(it.m, first, n, 4), local, m);
        load8<true>(chunk_of(it.v, first, n, 4), local, v);
    }
    if constexpr (!FULL && !G32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = e < left ? g[e] : 0.0f;
    }
    float root[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float gg = g[e] * h.grad_scale;
        m[e] = m[e] * b.beta1 + gg * b.one_minus_beta1;
        v[e] = v[e] * b.beta2 + (gg * gg) * b.one_minus_beta2;
    }
    sqrt8(v, root);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        p[e] = p[e] * h.decay - (m[e] / (root[e] * h.root_factor + b.eps)) * h.step_size;
    store8<FULL, P32>(it.param, i, left, p);
    if (it.copy) store8<FULL, false>(it.copy, i, left, p);
    if constexpr (S8) {
        uint32_t am = 0, av = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // elements past the end: 0 in m and v, whatever eps does to them
            // (a root's sign bit is set in a NaN only, which sorts on top either way)
            am = max_u(am, __float_as_uint(m[e]) & 0x7FFFFFFFu);
            av = max_u(av, __float_as_uint(root[e]));
        }
        const uint32_t cm = scale_of(block_max(am)), cv = scale_of(block_max(av));
        store_codes<FULL>(static_cast<uint8_t *>(it.m), i, left, encode8<SR, false>(m, cm, bits));
        store_codes<FULL>(static_cast<uint8_t *>(it.v), i, left, encode8<SR, true>(root, cv, bits));
        if ((FULL || left > 0) && (threadIdx.x & 3) == 0) {
            it.ms[i / 32] = (uint8_t)cm;
            it.vs[i / 32] = (uint8_t)cv;
        }
    } else {
        store8<FULL, true>(it.m, i, left, m);
        store8<FULL, true>(it.v, i, left, v);
    }
}

template <bool P32, bool G32, bool S8, bool SR, int ITEMS>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwTable<ITEMS> b) {
    // the tensor of this workgroup's chunk
    int t = 0;
    {
        int lo = 0, hi = b.count - 1;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (blockIdx.x < b.t[mid].chunk_end) hi = mid;
            else lo = mid + 1;
        }
        t = lo;
    }
    const AdamwItem &it = b.t[t];
    const int64_t first = (int64_t)(blockIdx.x - (t ? b.t[t - 1].chunk_end : 0u)) * kChunk;
    mx_adamw_step h = b.step;
    if (b.dev_step) h = *b.dev_step;
    if (first + kChunk <= it.numel) update8<true, P32, G32, S8, SR>(b, it, h, first, kChunk);
    else update8<false, P32, G32, S8, SR>(b, it, h, first, (int)(it.numel - first));
}

template <bool P32, bool G32, int ITEMS>
hipError_t launch_table(const AdamwTable<ITEMS> &b, bool s8, bool sr, unsigned blocks, hipStream_t stream) {
    auto kernel = !s8 ? adamw_kernel<P32, G32, false, false, ITEMS>
                      : (sr ? adamw_kernel<P32, G32, true, true, ITEMS> : adamw_kernel<P32, G32, true, false, ITEMS>);
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kThreads), 0, stream, b);
    return hipGetLastError();
}

// Tensors of a short table: three small tensors 4.7 us a step (5.2 with the long one).
constexpr int kFewItems = 6;

template <bool P32, bool G32>
hipError_t launch_states(const AdamwBatch &b, bool s8, bool sr, unsigned blocks, hipStream_t stream) {
    if (b.count > kFewItems) return launch_table<P32, G32>(b, s8, sr, blocks, stream);
    AdamwTable<kFewItems> few;
    memcpy(&few, &b, offsetof(AdamwBatch, t) + b.count * sizeof(AdamwItem));
    return launch_table<P32, G32>(few, s8, sr, blocks, stream);
}

}  // namespace

int64_t adamw_chunks(int64_t numel) { return cdiv(numel, kChunk); }

hipError_t launch_adamw(const AdamwBatch &b, bool p32, bool g32, bool s8, bool sr, hipStream_t stream) {
    const unsigned blocks = b.t[b.count - 1].chunk_end;
    if (p32) return g32 ? launch_states<true, true>(b, s8, sr, blocks, stream)
                        : launch_states<true, false>(b, s8, sr, blocks, stream);
    return g32 ? launch_states<false, true>(b, s8, sr, blocks, stream)
               : launch_states<false, false>(b, s8, sr, blocks, stream);
}

}  // namespace mx
