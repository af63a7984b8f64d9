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
// for training.  A positive sqrt(v) keeps at least the smallest code: at 0
// the next update would be divided by eps.
//
// Bound by memory (26 bytes per element with fp32 states, 14.125 with 8-bit
// ones at fp32 parameters and bf16 gradients).  A lane owns 8 consecutive
// elements, so a block's largest value is found in its 4 lanes with two DPP
// quad permutes.

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

// Eight elements at p + i, of which the first `left` exist (the others read 0).
template <bool F32>
__device__ __forceinline__ void load8(const void *p, int64_t i, int left, float (&v)[8]) {
    if constexpr (F32) {
        const float *s = static_cast<const float *>(p) + i;
        if (left >= 8) {
            const f4_t a = __builtin_nontemporal_load(reinterpret_cast<const f4_t *>(s));
            const f4_t b = __builtin_nontemporal_load(reinterpret_cast<const f4_t *>(s) + 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < left ? s[e] : 0.0f;
        }
    } else {
        const uint16_t *s = static_cast<const uint16_t *>(p) + i;
        if (left >= 8) {
            const u4_t a = __builtin_nontemporal_load(reinterpret_cast<const u4_t *>(s));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(a[e] << 16);
                v[2 * e + 1] = __uint_as_float(a[e] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < left ? __uint_as_float((uint32_t)s[e] << 16) : 0.0f;
        }
    }
}

template <bool F32>
__device__ __forceinline__ void store8(void *p, int64_t i, int left, const float (&v)[8]) {
    if constexpr (F32) {
        float *s = static_cast<float *>(p) + i;
        if (left >= 8) {
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
        if (left >= 8) {
            __builtin_nontemporal_store(u4_t{w[0], w[1], w[2], w[3]}, reinterpret_cast<u4_t *>(s));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) s[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// Eight E4M3 codes at p + i (a multiple of 8) and their block's scale byte.
__device__ __forceinline__ void load_codes(const uint8_t *p, const uint8_t *scale, int64_t i, int left, u2_t &w,
                                           uint32_t &c) {
    w = u2_t{0u, 0u};
    c = 0;
    if (left <= 0) return;
    c = scale[i / 32];
    if (left >= 8) {
        w = __builtin_nontemporal_load(reinterpret_cast<const u2_t *>(p + i));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) w[e >> 2] |= (uint32_t)p[i + e] << (8 * (e & 3));
    }
}

// The values they stand for: E4M3 times 2^(c - 127), NaN for c = 0xFF.
__device__ __forceinline__ void decode8(u2_t w, uint32_t c, float (&v)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
        const f2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
        v[4 * h] = a[0]; v[4 * h + 1] = a[1]; v[4 * h + 2] = b[0]; v[4 * h + 3] = b[1];
    }
    const int e = c == 0xFFu ? 0 : (int)c - 127;
    const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = c == 0xFFu ? nan : __builtin_ldexpf(v[k], e);
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

// Eight values -> E4M3 codes under scale byte c.  u = |x| 2^(7 - c) as an
// fp32 pattern has E4M3's fields on top (its subnormal step falls on the fp32
// subnormal grid): the code is u >> 20, plus 1 when the 16 bits below it
// exceed what the random bits leave (SR) or by the nearest-even rule.
template <bool SR, bool ROOT>
__device__ __forceinline__ u2_t encode8(const float (&x)[8], uint32_t c, const uint32_t (&bits)[8]) {
    u2_t w = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t xb = __float_as_uint(x[e]);
        const uint32_t u = __float_as_uint(__builtin_ldexpf(__uint_as_float(xb & 0x7FFFFFFFu), 7 - (int)c));
        uint32_t code = SR ? (u + ((ROOT ? bits[e] >> 16 : bits[e] & 0xFFFFu) << 4)) >> 20
                           : (u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20;
        code = code < 126u ? code : 126u;
        if (ROOT) code = x[e] > 0.0f && code == 0u ? 1u : code;
        else code |= (xb >> 24) & 0x80u;
        w[e >> 2] |= code << (8 * (e & 3));
    }
    return c == 0xFFu ? u2_t{0u, 0u} : w;
}

__device__ __forceinline__ void store_codes(uint8_t *p, int64_t i, int left, u2_t w) {
    if (left >= 8) {
        __builtin_nontemporal_store(w, reinterpret_cast<u2_t *>(p + i));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) p[i + e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
    }
}

template <bool P32, bool G32, bool S8, bool SR>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwBatch b) {
#pragma clang fp contract(off)
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
    const uint32_t first = t ? b.t[t - 1].chunk_end : 0u;
    const int64_t i = (int64_t)(blockIdx.x - first) * kChunk + (int64_t)threadIdx.x * kLaneElems;
    const int64_t l = it.numel - i;
    const int left = l < 0 ? 0 : (l > 8 ? 8 : (int)l);
    mx_adamw_step h = b.step;
    if (b.dev_step) h = *b.dev_step;

    float p[8], g[8], m[8], v[8];
    load8<G32>(it.grad, i, left, g);
    load8<P32>(it.param, i, left, p);
    if constexpr (S8) {
        u2_t wm, wv;
        uint32_t cm, cv;
        load_codes(static_cast<const uint8_t *>(it.m), it.ms, i, left, wm, cm);
        load_codes(static_cast<const uint8_t *>(it.v), it.vs, i, left, wv, cv);
        decode8(wm, cm, m);
        decode8(wv, cv, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * v[e];
    } else {
        load8<true>(it.m, i, left, m);
        load8<true>(it.v, i, left, v);
    }
    float root[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float gg = g[e] * h.grad_scale;
        m[e] = m[e] * b.beta1 + gg * b.one_minus_beta1;
        v[e] = v[e] * b.beta2 + (gg * gg) * b.one_minus_beta2;
        root[e] = __builtin_sqrtf(v[e]);
        p[e] = p[e] * h.decay - (m[e] / (root[e] * h.root_factor + b.eps)) * h.step_size;
    }
    store8<P32>(it.param, i, left, p);
    if (it.copy) store8<false>(it.copy, i, left, p);
    if constexpr (S8) {
        uint32_t am = 0, av = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // elements past the end: 0 in m and v, whatever eps does to them
            am = max_u(am, __float_as_uint(m[e]) & 0x7FFFFFFFu);
            av = max_u(av, __float_as_uint(root[e]) & 0x7FFFFFFFu);
        }
        const uint32_t cm = scale_of(block_max(am)), cv = scale_of(block_max(av));
        uint32_t bits[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
        if constexpr (SR) {
            const uint64_t n = (uint64_t)i >> 2;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t c[4] = {(uint32_t)(n + q), (uint32_t)((n + q) >> 32), it.tensor_id, 4u};
                philox(c, (uint32_t)h.seed, (uint32_t)(h.seed >> 32));
#pragma unroll
                for (int e = 0; e < 4; ++e) bits[4 * q + e] = c[e];
            }
        }
        store_codes(static_cast<uint8_t *>(it.m), i, left, encode8<SR, false>(m, cm, bits));
        store_codes(static_cast<uint8_t *>(it.v), i, left, encode8<SR, true>(root, cv, bits));
        if (left > 0 && (threadIdx.x & 3) == 0) {
            it.ms[i / 32] = (uint8_t)cm;
            it.vs[i / 32] = (uint8_t)cv;
        }
    } else {
        store8<true>(it.m, i, left, m);
        store8<true>(it.v, i, left, v);
    }
}

template <bool P32, bool G32>
hipError_t launch_states(const AdamwBatch &b, bool s8, bool sr, unsigned blocks, hipStream_t stream) {
    auto kernel = !s8 ? adamw_kernel<P32, G32, false, false>
                      : (sr ? adamw_kernel<P32, G32, true, true> : adamw_kernel<P32, G32, true, false>);
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kThreads), 0, stream, b);
    return hipGetLastError();
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
