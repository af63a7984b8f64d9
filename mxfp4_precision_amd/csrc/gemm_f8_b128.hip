// FP8 products with one E8M0 scale for each block of 128 elements along K:
//   C[i][j] = sum_b 2^(sa[i][b]-127) 2^(sb[j][b]-127) sum_{k in block b} a[i][k] b[j][k]  (+ bias[j])
// on the tiled FP8 blobs of mx_quantize_fp8_b128, E4M3 or E5M2 elements, fp32
// accumulation, bf16 (nearest even) or fp32 output.  The scales are powers of
// two, so the matrix instruction applies them itself: V_MFMA_SCALE takes a
// scale for each 32 elements of a row, and a block of 128 gives it the same
// byte four times.  (A scale of fp32 would have to be applied to each block's
// partial sums by 16 vector FMAs for every 128 matrix cycles.)
//
// The instruction does not sum FP8 products in full: it truncates each to a
// multiple of 2^-13 of the largest of its group of 8 along k, then adds in
// fp32; a bf16 result rounds 16 times more coarsely.
//
// Tiled form.  An atom is 16 rows x 64 elements (1 KB), a tile's k-step of 64
// elements its row groups' atoms, fetched into LDS by DMA and read back as
// operands of V_MFMA_SCALE_F32_32X32X64 (32 bytes a lane: two 16-byte slices
// of an atom).  What LDS delivers decides the shape: a CU's matrix pipes take
// 1024 cycles for one k-step of a 256x256 tile, and LDS 256 to receive it and 8
// for each KB read: with 8 waves of 128x64 that is 768 to read (as much as the
// pipes in all), with 4 waves of 128x128 512.  So a wave holds 128x128 of C (256
// accumulators a lane, one wave per SIMD), and hides its own latencies: each
// k-step is kSlots slots of one MFMA, one or two operand reads of the next step
// and the DMA instructions of the step three ahead, in fixed order.

#include "f8_b128.h"
#include "gemm_f8_b128_forms.h"
#include "gemm_pipeline.h"

namespace mx {
namespace {

// What the shared LDS and epilogue helpers need to know of a shape.
template <class S>
struct F8Cfg {
    static constexpr int kStages = 4;
    static constexpr int kBM = S::kBM, kBN = S::kBN, kWM = S::kWM, kWN = S::kWN, kKG = 1;
    static constexpr int kWaves = S::kWaves, kWavesM = S::kWavesM, kThreads = S::kThreads;
    static constexpr int kGA = kBM / 16, kGB = kBN / 16, kAtoms = kGA + kGB;   // atoms per k-step
    static constexpr int kTA = kWM / 16, kTB = kWN / 16;
    static constexpr int kMA = kWM / 32, kMB = kWN / 32;
    static constexpr int kSlots = kMA * kMB;               // MFMAs per wave and k-step
    static constexpr int kStageBytes = kAtoms * 1024;
    static constexpr int kLoads = kAtoms / kWaves;         // DMA instructions per wave and k-step
    static constexpr int kScaleLoads = kAtoms / 4 / kWaves;   // ... per 8 k-steps (a unit: 4 scale atoms of 64 bytes)
    static constexpr int kReads = 2 * (kMA + kMB);         // operand reads per wave and k-step
    static_assert(kAtoms % (4 * kWaves) == 0 && kGA % kWaves == 0 && kGA % 4 == 0, "whole DMA units");
};
using F8Main = F8Cfg<Shape<256, 256, 128, 128, 1>>;
using F8Small = F8Cfg<Shape<128, 128, 64, 64, 1>>;

template <class C>
__device__ __forceinline__ uint8_t *f8_scales(int which) {
    return g_lds<2 * C::kAtoms * 64, 4> + which * (C::kAtoms * 64);
}

// STREAM: the workgroup runs several tiles back to back as one stream of
// k-steps, a tile taking `steps` of them; a DMA for step steps + j fetches step j
// of the next tile (*_next; kleft = its k-steps, 0 when there is none).
template <class C, bool STREAM>
struct F8Ctx {
    static constexpr bool kStream = STREAM;
    __amdgpu_buffer_rsrc_t rA, rB, rAs, rBs, rBias;
    int row[C::kLoads];            // byte offsets of this wave's atoms at k-step 0 (wave-uniform)
    uint32_t sc[C::kScaleLoads];   // per lane: byte offsets of its scale words at k-group 0
    int ksteps, kgroups, wave, lane16;
    int row_next[STREAM ? C::kLoads : 1];
    uint32_t sc_next[STREAM ? C::kScaleLoads : 1];
    int steps, kleft;
    uint32_t bias;                 // per lane: byte offset of its two bias values
    int parity;                    // scale buffer of the tile's k-group 0
};

template <class C>
struct F8Regs {
    v8i a[2][C::kMA], b[2][C::kMB];   // operands of even and odd k-steps
    uint32_t sa[C::kMA], sb[C::kMB];  // scales: byte (k-step % 8) / 2
    uint32_t sa_n[C::kMA], sb_n[C::kMB];
};

// DMA instruction V of k-step k into stage S, or (V >= kLoads) of the scales of
// k-group h.  Past K the lane offset is out of range, which gives zeros; the
// scalar one then stays inside (the range check subtracts it from the range).
template <class C, int S, int V, class X>
__device__ __forceinline__ void f8_dma(const X &c, int k) {
    // (hidden, so that the addresses of all stages are not held in registers)
    int w = c.wave;
    asm volatile("" : "+s"(w));
    const int a = C::kWaves * V + w;
    constexpr bool isA = C::kWaves * (V + 1) <= C::kGA;
    const __amdgpu_buffer_rsrc_t rsrc = isA ? c.rA : c.rB;
    bool in = k < c.ksteps;
    int row = c.row[V];
    if constexpr (X::kStream) {
        if (k >= c.steps) {
            k -= c.steps;
            in = k < c.kleft;
            row = c.row_next[V];
        }
    }
    const uint32_t voff = in ? (uint32_t)c.lane16 : kOutOfRange;
    const uint32_t soff = (uint32_t)row + (in ? (uint32_t)k * 1024u : 0u);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, MX_LDS((stage_buf<C, S, 0>() + a * 1024)), 16, voff, soff, 0, 0);
}
template <class C, int V, class X>
__device__ __forceinline__ void f8_dma_scale(const X &c, int h) {
    const int u = C::kWaves * V + c.wave, to = (h + c.parity) & 1;
    const bool isA = 4 * u < C::kGA;   // wave-uniform
    const __amdgpu_buffer_rsrc_t rsrc = isA ? c.rAs : c.rBs;
    uint32_t voff = h < c.kgroups ? c.sc[V] + (uint32_t)h * 64u : kOutOfRange;
    if constexpr (X::kStream)
        if (8 * h >= c.steps) voff = c.kleft > 0 ? c.sc_next[V] : kOutOfRange;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, MX_LDS((f8_scales<C>(to) + u * 256)), 4, voff, 0, 0, 0);
}
template <class C, int S, int V = 0, class X>
__device__ __forceinline__ void f8_dma_step(const X &c, int k) {
    if constexpr (V < C::kLoads) {
        f8_dma<C, S, V>(c, k);
        f8_dma_step<C, S, V + 1>(c, k);
    }
}
template <class C, int V = 0, class X>
__device__ __forceinline__ void f8_dma_scales(const X &c, int h) {
    if constexpr (V < C::kScaleLoads) {
        f8_dma_scale<C, V>(c, h);
        f8_dma_scales<C, V + 1>(c, h);
    }
}

// Operand read R (in order of first use: b[0], a[0..], b[1..], two halves
// each) from stage S into set P.
template <class C, int S, int P, int R>
__device__ __forceinline__ void f8_read(F8Regs<C> &r, int off_a, int off_b) {
    constexpr int q = R / 2, half = R % 2;
    constexpr bool isB = q == 0 || q > C::kMA;
    constexpr int t = q == 0 ? 0 : (isB ? q - C::kMA : q - 1);
    const v4u_t v = *reinterpret_cast<const v4u_t *>(stage_buf<C, S, 0>() + (isB ? off_b : off_a) + 2 * t * 1024 +
                                                     half * 256);
    v8i &d = isB ? r.b[P][t] : r.a[P][t];
#pragma unroll
    for (int e = 0; e < 4; ++e) d[4 * half + e] = (int)v[e];
}
template <class C, int S, int P, int R0, int R1>
__device__ __forceinline__ void f8_reads(F8Regs<C> &r, int off_a, int off_b) {
    if constexpr (R0 < R1) {
        f8_read<C, S, P, R0>(r, off_a, off_b);
        f8_reads<C, S, P, R0 + 1, R1>(r, off_a, off_b);
    }
}

struct F8Off {
    int a, b, sa, sb;   // LDS byte offsets of this lane's first A and B operands and scale words
};

// LDS of a wave's bias values (stream form).
template <class C>
__device__ __forceinline__ uint8_t *f8_bias(int wave) {
    return g_lds<C::kWaves * 256, 5> + wave * 256;
}

// Slot T of the k-step with position SG of 8: the MFMA, the reads of the next
// step's operands that fall to it, the DMA instructions of step k + 3, and at
// the end of a group of 8 the next group's scales.  FRESH: a tile's first group
// in the stream form, whose first step starts the accumulators from 0 and which
// fetches the tile's bias.
template <class C, int FA, int FB, int SG, bool FRESH, int T, class X>
__device__ __forceinline__ void f8_slot(const X &c, int k, v16f (&acc)[C::kMB][C::kMA], F8Regs<C> &r,
                                        const F8Off &o) {
    constexpr int i = T / C::kMA, j = T % C::kMA, P = SG & 1, S = SG & 3;
    // (plain-typed locals: a builtin call on template-dependent operands does
    // not resolve in the host compilation pass)
    const v8i bop = r.b[P][i], aop = r.a[P][j];
    const int sb = (int)r.sb[i], sa = (int)r.sa[j];
    const v16f cin = FRESH && SG == 0 ? v16f{} : acc[i][j];
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bop, aop, cin, FB, FA, SG / 2, sb, SG / 2, sa);
    f8_reads<C, (S + 1) & 3, P ^ 1, T * C::kReads / C::kSlots, (T + 1) * C::kReads / C::kSlots>(r, o.a, o.b);
    if constexpr (SG == 7 && T < C::kMA) {
        const uint8_t *s = f8_scales<C>((k / 8 + 1 + c.parity) & 1);
        r.sa_n[T] = *reinterpret_cast<const uint32_t *>(s + o.sa + T * 128);
        if constexpr (T < C::kMB) r.sb_n[T] = *reinterpret_cast<const uint32_t *>(s + o.sb + T * 128);
    }
    constexpr int d0 = T * C::kLoads / C::kSlots, d1 = (T + 1) * C::kLoads / C::kSlots;
    if constexpr (d1 > d0) f8_dma<C, (S + 3) & 3, d0>(c, k + 3);
    if constexpr (d1 > d0 + 1) f8_dma<C, (S + 3) & 3, d0 + 1>(c, k + 3);
    static_assert(d1 <= d0 + 2, "DMA instructions per slot");
    if constexpr (SG == 4 && T < C::kScaleLoads) f8_dma_scale<C, T>(c, k / 8 + 1);
    if constexpr (FRESH && SG == 4 && T == C::kScaleLoads) {
        const __amdgpu_buffer_rsrc_t rsrc = c.rBias;
        const uint32_t voff = c.bias;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, MX_LDS(f8_bias<C>(c.wave)), 4, voff, 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}
template <class C, int FA, int FB, int SG, bool FRESH, int T = 0, class X>
__device__ __forceinline__ void f8_slots(const X &c, int k, v16f (&acc)[C::kMB][C::kMA], F8Regs<C> &r, const F8Off &o) {
    if constexpr (T < C::kSlots) {
        f8_slot<C, FA, FB, SG, FRESH, T>(c, k, acc, r, o);
        f8_slots<C, FA, FB, SG, FRESH, T + 1>(c, k, acc, r, o);
    }
}

// Stores that a wave issues for a tile in the stream form.
template <class C>
__host__ __device__ constexpr int f8_stores() {
    return C::kWM * C::kWN * 2 / 1024;
}

// Vector memory instructions that may be outstanding at the start of the step
// at position SG: all that were issued after its next step's DMA, that is step
// k - 1's (and at positions 0 and 1 of a FRESH group the previous tile's stores,
// which were issued between).
template <class C>
constexpr int f8_outstanding(int SG, bool fresh) {
    return C::kLoads + (SG == 5 ? C::kScaleLoads + (fresh ? 1 : 0) : 0) + (fresh && SG < 2 ? f8_stores<C>() : 0);
}

// K-steps k0 .. k0 + 7, or (one tile) fewer at the end of K, a multiple of two.
template <class C, int FA, int FB, bool FRESH, int SG = 0, class X>
__device__ __forceinline__ void f8_group(const X &c, int k0, v16f (&acc)[C::kMB][C::kMA], F8Regs<C> &r,
                                         const F8Off &o) {
    if constexpr (SG < 8) {
        if constexpr (!X::kStream && SG > 0 && SG % 2 == 0)
            if (k0 + SG >= c.ksteps) return;
        // Step k + 1 has landed for this wave and, past the barrier, for all; and
        // every wave is past step k - 1, so the stage that step k + 3 goes to
        // (step k - 1's, read during step k - 2) is free.
        static_assert(f8_outstanding<C>(SG, FRESH) <= 63, "vmcnt range");
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(f8_outstanding<C>(SG, FRESH)) : "memory");
        __builtin_amdgcn_sched_barrier(0);
        f8_slots<C, FA, FB, SG, FRESH>(c, k0 + SG, acc, r, o);
        if constexpr (SG == 7) {
#pragma unroll
            for (int t = 0; t < C::kMA; ++t) r.sa[t] = r.sa_n[t];
#pragma unroll
            for (int t = 0; t < C::kMB; ++t) r.sb[t] = r.sb_n[t];
        }
        f8_group<C, FA, FB, FRESH, SG + 1>(c, k0, acc, r, o);
    }
}

// Scales of k-group 0 and operands of step 0, once they have landed.
template <class C>
__device__ __forceinline__ void f8_first(F8Regs<C> &r, const F8Off &o) {
    const uint8_t *s = f8_scales<C>(0);
#pragma unroll
    for (int t = 0; t < C::kMA; ++t) r.sa[t] = *reinterpret_cast<const uint32_t *>(s + o.sa + t * 128);
#pragma unroll
    for (int t = 0; t < C::kMB; ++t) r.sb[t] = *reinterpret_cast<const uint32_t *>(s + o.sb + t * 128);
    f8_reads<C, 0, 0, 0, C::kReads>(r, o.a, o.b);
}

template <class C>
__device__ __forceinline__ F8Off f8_offsets(int wave, int lane) {
    const int wm = wave % C::kWavesM, wn = wave / C::kWavesM;
    const int lrow = lane & 31, lhi = lane >> 5;
    const int frag = (lrow >> 4) * 1024 + ((lrow & 15) + 32 * lhi) * 16, word = (lrow >> 4) * 64 + (lrow & 15) * 4;
    F8Off o = {frag + wm * C::kTA * 1024, frag + (C::kGA + wn * C::kTB) * 1024, word + wm * C::kTA * 64,
               word + (C::kGA + wn * C::kTB) * 64};
    // hide the offsets' known zero bits, so that constants go to the instructions' offset field
    asm volatile("" : "+v"(o.a), "+v"(o.b), "+v"(o.sa), "+v"(o.sb));
    return o;
}

// Offsets of a tile's atoms and scale words.  Row groups past an operand are
// clamped to its last one: those rows of C are not stored.
template <class C>
__device__ __forceinline__ void f8_tile_rows(int tm, int tn, int nGA, int nGB, int ksteps, int kgroups, int wave,
                                             int lane, int (&row)[C::kLoads], uint32_t (&sc)[C::kScaleLoads]) {
    const auto group_of = [&](int a) {
        return a < C::kGA ? min(tm * C::kGA + a, nGA - 1) : min(tn * C::kGB + (a - C::kGA), nGB - 1);
    };
#pragma unroll
    for (int v = 0; v < C::kLoads; ++v) row[v] = group_of(C::kWaves * v + wave) * ksteps * 1024;
#pragma unroll
    for (int v = 0; v < C::kScaleLoads; ++v)
        sc[v] = (uint32_t)(group_of(4 * (C::kWaves * v + wave) + (lane >> 4)) * kgroups * 64 + 4 * (lane & 15));
}

template <class C, int FA, int FB, bool OUT_BF16>
__global__ __launch_bounds__(C::kThreads) void gemm_f8_b128_kernel(int64_t M, int64_t N, int64_t K_pad, int tiles_m,
                                                                   int tiles_n, int group_m,
                                                                   const uint8_t *__restrict__ A,
                                                                   const uint8_t *__restrict__ As,
                                                                   const uint8_t *__restrict__ B,
                                                                   const uint8_t *__restrict__ Bs,
                                                                   const uint16_t *__restrict__ bias,
                                                                   void *__restrict__ Cout, int64_t ldc) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave / C::kWavesM;
    int tm, tn;
    tile_of(blockIdx.x, gridDim.x, tiles_m, tiles_n, group_m, tm, tn);

    F8Ctx<C, false> c;
    c.ksteps = (int)(K_pad / 64);
    c.kgroups = (int)cdiv(K_pad, 512);
    c.wave = wave;
    c.lane16 = lane * 16;
    c.parity = 0;
    const int nGA = (int)cdiv(M, 16), nGB = (int)cdiv(N, 16);
    c.rA = make_rsrc(A, (int64_t)nGA * c.ksteps * 1024);
    c.rB = make_rsrc(B, (int64_t)nGB * c.ksteps * 1024);
    c.rAs = make_rsrc(As, (int64_t)nGA * c.kgroups * 64);
    c.rBs = make_rsrc(Bs, (int64_t)nGB * c.kgroups * 64);
    f8_tile_rows<C>(tm, tn, nGA, nGB, c.ksteps, c.kgroups, wave, lane, c.row, c.sc);

    v16f acc[C::kMB][C::kMA];
#pragma unroll
    for (int i = 0; i < C::kMB; ++i)
#pragma unroll
        for (int j = 0; j < C::kMA; ++j) acc[i][j] = v16f{};

    const F8Off o = f8_offsets<C>(wave, lane);
    f8_dma_scales<C>(c, 0);
    f8_dma_step<C, 0>(c, 0);
    f8_dma_step<C, 1>(c, 1);
    f8_dma_step<C, 2>(c, 2);
    F8Regs<C> r;
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(2 * C::kLoads) : "memory");
    f8_first<C>(r, o);
    for (int k0 = 0; k0 < c.ksteps; k0 += 8) f8_group<C, FA, FB, false>(c, k0, acc, r, o);
    // drain the trailing (out-of-range) DMAs before LDS is reused
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    if (bias) {
        v2u_t bits[C::kMB * 4];
        load_bias<C>(make_rsrc(bias, cdiv(N * 2, 16) * 16), tn, wn, lane, bits);
        add_bias<C>(acc, bits);
    }
    store_tile<C, OUT_BF16>(acc, tm, tn, M, N, Cout, ldc, 0, wave, wave, lane);
}

// Persistent form (bf16 output): one workgroup per CU runs tiles b, b +
// gridDim.x, ... of the tile order as one stream of k-steps.  A tile takes
// `steps` = its k-steps rounded up to a multiple of 8; its last steps fetch the
// next tile's first three, their scales and its first operands, so nothing
// drains between tiles.  The epilogue stages C through stage 3 (the others hold
// the next tile's steps), 8 KB a wave: in pass p a wave writes its MFMA row tile
// p (32 rows x 128 columns, 16-byte chunk c of row r at c ^ r % 16) and reads it
// back as whole 256-byte row segments, 4 rows per store.  Every wave issues
// f8_stores() stores a tile whatever the edges (what lies outside C has an
// offset out of range), so that the next tile's first two waits can count past
// them; the third needs them done.  Needs N % 8 == 0 and 32-bit offsets into C.
template <class C, bool BIAS>
__device__ __forceinline__ void f8_store_private(const v16f (&acc)[C::kMB][C::kMA], int tm, int tn, int M, int N,
                                                 __amdgpu_buffer_rsrc_t rC, int ldc, int wave, int lane) {
    constexpr int kSlot = 32 * C::kWN * 2;
    static_assert(C::kWN == 128 && kSlot * C::kWaves == C::kStageBytes, "one slot per wave fills stage 3");
    // (hidden, so that no address is computed ahead of the tile loop and held)
    asm volatile("" : "+v"(lane), "+s"(wave));
    const int wm = wave % C::kWavesM, wn = wave / C::kWavesM;
    const int lrow = lane & 31, lhi = lane >> 5;
    const int row0 = tm * C::kBM + C::kWM * wm + (lane >> 4), col = tn * C::kBN + C::kWN * wn + 8 * (lane & 15);
    uint8_t *slot = stage_buf<C, 3, 0>() + wave * kSlot;
    const uint8_t *b = f8_bias<C>(wave) + 8 * lhi;
    // every wave is done reading stage 3 (a bare barrier: a fence would also
    // wait for the next tile's DMAs)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int p = 0; p < C::kMA; ++p) {
#pragma unroll
        for (int i = 0; i < C::kMB; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][p][4 * q + e];
                if constexpr (BIAS) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(b + 2 * (32 * i + 8 * q));
                    v[0] += __uint_as_float(w.x << 16);
                    v[1] += __uint_as_float(w.x & 0xFFFF0000u);
                    v[2] += __uint_as_float(w.y << 16);
                    v[3] += __uint_as_float(w.y & 0xFFFF0000u);
                }
                *reinterpret_cast<uint2 *>(slot + lrow * 256 + (((4 * i + q) ^ (lrow & 15)) * 16) + 8 * lhi) =
                    uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            }
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const int r = 4 * s + (lane >> 4);
            const v4u_t v = *reinterpret_cast<const v4u_t *>(slot + r * 256 + (((lane & 15) ^ (r & 15)) * 16));
            const int row = row0 + 32 * p + 4 * s;
            const uint32_t off =
                row < M && col < N ? ((uint32_t)row * (uint32_t)ldc + (uint32_t)col) * 2u : kOutOfRange;
            __builtin_amdgcn_raw_buffer_store_b128(v, rC, off, 0, kCachePolicyNT);
        }
    }
}

template <class C, int FA, int FB, bool BIAS>
__global__ __launch_bounds__(C::kThreads) void gemm_f8_b128_stream_kernel(int M, int N, int K_pad, int tiles_m,
                                                                          int tiles_n, int group_m,
                                                                          const uint8_t *__restrict__ A,
                                                                          const uint8_t *__restrict__ As,
                                                                          const uint8_t *__restrict__ B,
                                                                          const uint8_t *__restrict__ Bs,
                                                                          const uint16_t *__restrict__ bias,
                                                                          void *__restrict__ Cout, int ldc) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave / C::kWavesM;
    const int P = gridDim.x, tiles = tiles_m * tiles_n;
    F8Ctx<C, true> c;
    c.ksteps = K_pad / 64;
    c.kgroups = (K_pad + 511) / 512;
    c.steps = 8 * c.kgroups;
    c.wave = wave;
    c.lane16 = lane * 16;
    c.parity = 0;
    const int nGA = (M + 15) / 16, nGB = (N + 15) / 16;
    c.rA = make_rsrc(A, (int64_t)nGA * c.ksteps * 1024);
    c.rB = make_rsrc(B, (int64_t)nGB * c.ksteps * 1024);
    c.rAs = make_rsrc(As, (int64_t)nGA * c.kgroups * 64);
    c.rBs = make_rsrc(Bs, (int64_t)nGB * c.kgroups * 64);
    // whole 16-byte blocks, as the range check zeroes whole dwords
    c.rBias = make_rsrc(bias, BIAS ? ((int64_t)N * 2 + 15) / 16 * 16 : 0);
    const __amdgpu_buffer_rsrc_t rC = make_rsrc(Cout, ((int64_t)(M - 1) * ldc + N) * 2);

    int vb = blockIdx.x, tm, tn, tm_next = 0, tn_next = 0;
    const auto look_ahead = [&]() {
        c.kleft = 0;
        if (vb + P < tiles) {
            tile_of(vb + P, tiles, tiles_m, tiles_n, group_m, tm_next, tn_next);
            f8_tile_rows<C>(tm_next, tn_next, nGA, nGB, c.ksteps, c.kgroups, wave, lane, c.row_next, c.sc_next);
            c.kleft = c.ksteps;
        }
    };
    tile_of(vb, tiles, tiles_m, tiles_n, group_m, tm, tn);
    f8_tile_rows<C>(tm, tn, nGA, nGB, c.ksteps, c.kgroups, wave, lane, c.row, c.sc);
#pragma unroll
    for (int v = 0; v < C::kLoads; ++v) c.row_next[v] = c.row[v];
#pragma unroll
    for (int v = 0; v < C::kScaleLoads; ++v) c.sc_next[v] = c.sc[v];
    look_ahead();

    const F8Off o = f8_offsets<C>(wave, lane);
    f8_dma_scales<C>(c, 0);
    f8_dma_step<C, 0>(c, 0);
    f8_dma_step<C, 1>(c, 1);
    f8_dma_step<C, 2>(c, 2);
    F8Regs<C> r;
    // all of it, so that the first tile's first two waits, which count past
    // stores that it does not have, need not wait; as a builtin, so that the
    // compiler's own wait tracking knows too
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    __builtin_amdgcn_s_barrier();
    f8_first<C>(r, o);
    v16f acc[C::kMB][C::kMA];
    for (;;) {
        c.bias = (uint32_t)(tn * C::kBN + wn * C::kWN + 2 * lane) * 2u;
        f8_group<C, FA, FB, true>(c, 0, acc, r, o);
        for (int k0 = 8; k0 < c.steps; k0 += 8) f8_group<C, FA, FB, false>(c, k0, acc, r, o);
        f8_store_private<C, BIAS>(acc, tm, tn, M, N, rC, ldc, wave, lane);
        vb += P;
        if (vb >= tiles) break;
        tm = tm_next;
        tn = tn_next;
#pragma unroll
        for (int v = 0; v < C::kLoads; ++v) c.row[v] = c.row_next[v];
#pragma unroll
        for (int v = 0; v < C::kScaleLoads; ++v) c.sc[v] = c.sc_next[v];
        c.parity ^= c.kgroups & 1;
        look_ahead();
    }
    // drain the stores and the trailing (out-of-range) DMAs
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// ------------------------------------------------------------ few rows
// Products of few rows (decoding, small training steps): what counts is reading
// the operands once and the latency of one pass, so nothing goes through LDS
// before the sums.  Two atoms of a row group are the operand of
// V_MFMA_SCALE_F32_16X16X128 (lane L: row L % 16, slice L / 16 of each atom; both
// operands take their k in the same order, and the scale is the same for all
// 128).  A workgroup's tile is MA x 16 rows x 16 NB columns.  Its waves split K:
// wave w takes block w % 4 of every (WAVES / 4)-th k-group from w / 4 on, so it
// uses one byte of each scale word, and the sums are added in wave order through
// LDS.
template <int FA, int FB, int MA, int NB, int WAVES, int DEPTH>
__device__ __forceinline__ void f8_few_sum(__amdgpu_buffer_rsrc_t rA, __amdgpu_buffer_rsrc_t rAs,
                                           __amdgpu_buffer_rsrc_t rB, __amdgpu_buffer_rsrc_t rBs, int gA0, int nGA,
                                           int gB0, int nGB, int kblocks, int kgroups, int ends, int wave,
                                           int lane, v4f (&acc)[MA][NB], int h0 = 0) {
    int a_row[MA], b_row[NB];
#pragma unroll
    for (int i = 0; i < MA; ++i) a_row[i] = min(gA0 + i, nGA - 1);
#pragma unroll
    for (int j = 0; j < NB; ++j) b_row[j] = min(gB0 + j, nGB - 1);
    const uint32_t lane16 = (uint32_t)lane * 16, word = (uint32_t)(lane & 15) * 4;
    constexpr int kStep = WAVES / 4;
    const int shift = 8 * (wave & 3);
    for (; h0 + kStep * DEPTH <= ends; h0 += kStep * DEPTH) {   // ends: kgroups rounded up to whole steps
        v4u_t a[DEPTH][MA][2], b[DEPTH][NB][2];
        uint32_t as[DEPTH][MA], bs[DEPTH][NB];
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            const int h = h0 + kStep * u + (wave >> 2), kb = 4 * h + (wave & 3);
            const bool in = kb < kblocks;   // past K: zeros, of data and scales (see f8_dma)
            const uint32_t off = in ? lane16 : kOutOfRange, soff = in ? word : kOutOfRange;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int at = in ? (b_row[j] * kblocks + kb) * 2048 : 0;
                b[u][j][0] = __builtin_amdgcn_raw_buffer_load_b128(rB, off, at, 0);
                b[u][j][1] = __builtin_amdgcn_raw_buffer_load_b128(rB, off + 1024, at, 0);
                bs[u][j] = __builtin_amdgcn_raw_buffer_load_b32(rBs, soff, in ? (b_row[j] * kgroups + h) * 64 : 0, 0);
            }
#pragma unroll
            for (int i = 0; i < MA; ++i) {
                const int at = in ? (a_row[i] * kblocks + kb) * 2048 : 0;
                a[u][i][0] = __builtin_amdgcn_raw_buffer_load_b128(rA, off, at, 0);
                a[u][i][1] = __builtin_amdgcn_raw_buffer_load_b128(rA, off + 1024, at, 0);
                as[u][i] = __builtin_amdgcn_raw_buffer_load_b32(rAs, soff, in ? (a_row[i] * kgroups + h) * 64 : 0, 0);
            }
        }
#pragma unroll
        for (int u = 0; u < DEPTH; ++u)
#pragma unroll
            for (int i = 0; i < MA; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const v8i bop = {(int)b[u][j][0][0], (int)b[u][j][0][1], (int)b[u][j][0][2], (int)b[u][j][0][3],
                                     (int)b[u][j][1][0], (int)b[u][j][1][1], (int)b[u][j][1][2], (int)b[u][j][1][3]};
                    const v8i aop = {(int)a[u][i][0][0], (int)a[u][i][0][1], (int)a[u][i][0][2], (int)a[u][i][0][3],
                                     (int)a[u][i][1][0], (int)a[u][i][1][1], (int)a[u][i][1][2], (int)a[u][i][1][3]};
                    const int sb = (int)(bs[u][j] >> shift), sa = (int)(as[u][i] >> shift);
                    const v4f cin = acc[i][j];
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bop, aop, cin, FB, FA, 0, sb, 0, sa);
                }
    }
    if constexpr (DEPTH > 1)
        f8_few_sum<FA, FB, MA, NB, WAVES, DEPTH / 2>(rA, rAs, rB, rBs, gA0, nGA, gB0, nGB, kblocks, kgroups, ends, wave,
                                                     lane, acc, h0);
}

// The waves' sums, added in wave order and stored: lane L of tile (i, j)
// holds row 16 i + L % 16, columns 16 j + 4 (L / 16) + 0..3.
template <int MA, int NB, int WAVES, bool OUT_BF16>
__device__ __forceinline__ void f8_few_store(const v4f (&acc)[MA][NB], int64_t row0, int64_t col0, int64_t M,
                                             int64_t N, const uint16_t *bias, void *Cout, int64_t ldc, int wave,
                                             int lane) {
    __shared__ v4f s_sum[WAVES][MA * NB][64];
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) s_sum[wave][i * NB + j][lane] = acc[i][j];
    __syncthreads();
    for (int t = wave; t < MA * NB; t += WAVES) {
        v4f v = s_sum[0][t][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) {
            const v4f q = s_sum[w][t][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += q[e];
        }
        const int64_t row = row0 + 16 * (t / NB) + (lane & 15);
        const int64_t col = col0 + 16 * (t % NB) + 4 * (lane >> 4);
        if (row >= M || col >= N) continue;
        if (bias) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < N) v[e] += __uint_as_float((uint32_t)bias[col + e] << 16);
        }
        const int64_t at = row * ldc + col;
        if constexpr (OUT_BF16) {
            uint16_t *dst = static_cast<uint16_t *>(Cout) + at;
            const v2u_t w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            if (col + 3 < N) {
                *reinterpret_cast<v2u_t *>(dst) = w;
            } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (col + e < N) dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
            }
        } else {
            float *dst = static_cast<float *>(Cout) + at;
            if (col + 3 < N) {
                *reinterpret_cast<v4f *>(dst) = v;
            } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (col + e < N) dst[e] = v[e];
            }
        }
    }
}

template <int FA, int FB, int MA, int NB, int WAVES, bool OUT_BF16>
__global__ __launch_bounds__(64 * WAVES) void gemm_f8_b128_few_kernel(
    int64_t M, int64_t N, int kblocks, int tiles_n, const uint8_t *__restrict__ A, const uint8_t *__restrict__ As,
    const uint8_t *__restrict__ B, const uint8_t *__restrict__ Bs, const uint16_t *__restrict__ bias,
    void *__restrict__ Cout, int64_t ldc) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tn = blockIdx.x % tiles_n, tm = blockIdx.x / tiles_n;
    const int nGA = (int)cdiv(M, 16), nGB = (int)cdiv(N, 16), kgroups = (kblocks + 3) / 4;
    v4f acc[MA][NB];
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = v4f{};
    f8_few_sum<FA, FB, MA, NB, WAVES, MA * NB >= 4 ? 2 : 8 / (MA * NB)>(
        make_rsrc(A, (int64_t)nGA * kblocks * 2048), make_rsrc(As, (int64_t)nGA * kgroups * 64),
        make_rsrc(B, (int64_t)nGB * kblocks * 2048), make_rsrc(Bs, (int64_t)nGB * kgroups * 64), tm * MA, nGA,
        tn * NB, nGB, kblocks, kgroups, (kgroups + WAVES / 4 - 1) / (WAVES / 4) * (WAVES / 4), wave, lane, acc);
    f8_few_store<MA, NB, WAVES, OUT_BF16>(acc, (int64_t)tm * MA * 16, (int64_t)tn * NB * 16, M, N, bias, Cout, ldc,
                                          wave, lane);
}

// A linear layer on up to 16 rows in one launch: as the few-rows product, but a
// wave quantizes the blocks of x that it multiplies.  Lane L holds row L % 16's
// slice L / 16 of both halves of a block, so the block's maximum is a lane
// exchange away and the codes are the operand; every workgroup does so for itself
// (x is small and stays in the L2s), while its weights are on their way.  Eight
// waves split K: wave w takes block w % 4 of every other k-group from w / 4 on, two
// at a time.  In us, 4 waves with four in flight / 8 with two / 16 with two: 1 row
// 4096 x 4096 7.1 / 5.9 / 5.8, 16 rows 9.5 / 7.8 / 7.8, 1 row 1024 x 1024 3.0 / 2.9
// / 4.0.
constexpr int kLinearWaves = 8;
template <int FX, int FW, int DEPTH>
__device__ __forceinline__ void f8_linear_sum(const uint16_t *__restrict__ x, int64_t M, int64_t K, int64_t ldx,
                                              __amdgpu_buffer_rsrc_t rB, __amdgpu_buffer_rsrc_t rBs, int g,
                                              int kblocks, int kgroups, int ends, int wave, int lane, v4f &acc,
                                              int h0 = 0) {
    const uint32_t lane16 = (uint32_t)lane * 16, word = (uint32_t)(lane & 15) * 4;
    const int64_t r = lane & 15;
    constexpr int kStep = kLinearWaves / 4;
    const int shift = 8 * (wave & 3);
    for (; h0 + kStep * DEPTH <= ends; h0 += kStep * DEPTH) {   // ends: kgroups rounded up to whole steps
        v4u_t b[DEPTH][2];
        uint32_t bs[DEPTH];
        u4_t v[DEPTH][4];
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            const int h = h0 + kStep * u + (wave >> 2), kb = 4 * h + (wave & 3);
            const bool in = kb < kblocks;   // past K: zeros, of data and scales (see f8_dma)
            const uint32_t off = in ? lane16 : kOutOfRange;
            const int at = in ? (g * kblocks + kb) * 2048 : 0;
            b[u][0] = __builtin_amdgcn_raw_buffer_load_b128(rB, off, at, 0);
            b[u][1] = __builtin_amdgcn_raw_buffer_load_b128(rB, off + 1024, at, 0);
            bs[u] = __builtin_amdgcn_raw_buffer_load_b32(rBs, in ? word : kOutOfRange,
                                                           in ? (g * kgroups + h) * 64 : 0, 0);
        }
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            const int64_t k0 = 128 * (int64_t)(4 * (h0 + kStep * u + (wave >> 2)) + (wave & 3));
            const int64_t k = k0 + 16 * (lane >> 4);
            if (k0 + 128 <= K) {
#pragma unroll
                for (int w = 0; w < 4; ++w) v[u][w] = u4_t{};
                if (r < M) {
                    const u4_t *p = reinterpret_cast<const u4_t *>(x + r * ldx + k);
                    v[u][0] = p[0]; v[u][1] = p[1]; v[u][2] = p[8]; v[u][3] = p[9];
                }
            } else {
                u4_t lo[2], hi[2];
                load16(x, M, K, ldx, r, k, lo);
                load16(x, M, K, ldx, r, k + 64, hi);
                v[u][0] = lo[0]; v[u][1] = lo[1]; v[u][2] = hi[0]; v[u][3] = hi[1];
            }
        }
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < 16; ++w) m = max2(m, v[u][w >> 2][w & 3] & 0x7FFF7FFFu);
            m = max2_xor<16>(m);
            m = max2_xor<32>(m);
            const uint32_t c = scale_byte<FX>((m & 0xFFFFu) > (m >> 16) ? (m & 0xFFFFu) : (m >> 16));
            const float scale = scale_of(c);
            v8i aop;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const uint32_t q = encode4<FX>(v[u][w >> 1][(w & 1) * 2], v[u][w >> 1][(w & 1) * 2 + 1], scale);
                aop[w] = c == 0xFFu ? 0 : (int)q;
            }
            const v8i bop = {(int)b[u][0][0], (int)b[u][0][1], (int)b[u][0][2], (int)b[u][0][3],
                             (int)b[u][1][0], (int)b[u][1][1], (int)b[u][1][2], (int)b[u][1][3]};
            const int sb = (int)(bs[u] >> shift), sa = (int)c;
            const v4f cin = acc;
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bop, aop, cin, FW, FX, 0, sb, 0, sa);
        }
    }
    if constexpr (DEPTH > 1)
        f8_linear_sum<FX, FW, DEPTH / 2>(x, M, K, ldx, rB, rBs, g, kblocks, kgroups, ends, wave, lane, acc, h0);
}

template <int FX, int FW, bool OUT_BF16>
__global__ __launch_bounds__(64 * kLinearWaves) void linear_f8_b128_kernel(
    int64_t M, int64_t N, int64_t K, const uint16_t *__restrict__ x, int64_t ldx, const uint8_t *__restrict__ W,
    const uint8_t *__restrict__ Ws, const uint16_t *__restrict__ bias, void *__restrict__ y, int64_t ldy) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kblocks = (int)cdiv(K, 128), kgroups = (kblocks + 3) / 4, nGB = (int)cdiv(N, 16);
    const int gB0 = (int)blockIdx.x;
    v4f acc[1][1] = {};
    f8_linear_sum<FX, FW, 2>(x, M, K, ldx, make_rsrc(W, (int64_t)nGB * kblocks * 2048),
                             make_rsrc(Ws, (int64_t)nGB * kgroups * 64), gB0, kblocks, kgroups,
                             (kgroups + kLinearWaves / 4 - 1) / (kLinearWaves / 4) * (kLinearWaves / 4), wave, lane,
                             acc[0][0]);
    f8_few_store<1, 1, kLinearWaves, OUT_BF16>(acc, 0, 16 * (int64_t)gB0, M, N, bias, y, ldy, wave, lane);
}

template <int FX, int FW>
hipError_t launch_linear(const F8LinearArgs &a, hipStream_t stream) {
    const F8GemmArgs &g = a.g;
    const bool bf = g.out_dtype == MX_BF16;
    auto kernel = bf ? linear_f8_b128_kernel<FX, FW, true> : linear_f8_b128_kernel<FX, FW, false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)cdiv(g.N, 16)), dim3(64 * kLinearWaves), 0, stream, g.M, g.N, g.K, a.x,
                       a.ldx, g.B, g.Bs, g.bias, g.C, g.ldc);
    return hipGetLastError();
}

// K == 0: C[i][j] = 0, or bias[j].
template <typename T>
__global__ void f8_fill_kernel(T *Cout, int64_t M, int64_t N, int64_t ldc, const uint16_t *bias) {
    const int64_t n = M * N;
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x) {
        const int64_t j = e % N;
        const uint16_t b = bias ? bias[j] : (uint16_t)0;
        if constexpr (sizeof(T) == 2) Cout[(e / N) * ldc + j] = b;
        else Cout[(e / N) * ldc + j] = __uint_as_float((uint32_t)b << 16);
    }
}

// Tile rows per band of the tile order: 4 and 8 within 1% but for 8192 x 4096 x
// 1024 (37.8 us and 41.3), 16 up to 4% slower.
constexpr int kBandRows = 4;

template <int FA, int FB, bool OUT_BF16>
hipError_t launch_formats(const F8GemmArgs &a, hipStream_t stream) {
    const int64_t K_pad = padded(a.K);
    switch (f8_gemm_form(a, device_cu_count())) {
        case F8Form::kFewRows: {
            const int ma = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
            const int nb = ma == 1 ? 1 : 2;
            const int64_t tiles_n = cdiv(a.N, 16 * nb), tiles = cdiv(a.M, 16 * ma) * tiles_n;
            // Eight waves for the widest tile where no CU gets two of them (us, 4 waves /
            // 8: 64 x 4096 x 4096 8.7 / 7.3, 512 x 1024 x 8192 14.9 / 11.6, 333 x 712 x
            // 1000 4.8 / 4.6; with three tiles a CU, of which it then holds one at a time,
            // 333 x 4096 x 4096 15.1 / 18.6).  With one k-group half of them would idle
            // (712 x 1000 x 328 4.2 / 6.1), and for the small tiles four do as well (16 x
            // 4096 x 4096 5.0 / 5.25, 23 x 5000 x 2888 5.9 / 6.0, 32 x 4096 x 4096 6.5 /
            // 6.1).
            const bool wide = ma == 4 && K_pad > 512 && tiles <= device_cu_count();
            auto kernel = ma == 1   ? gemm_f8_b128_few_kernel<FA, FB, 1, 1, 4, OUT_BF16>
                          : ma == 2 ? gemm_f8_b128_few_kernel<FA, FB, 2, 2, 4, OUT_BF16>
                          : wide    ? gemm_f8_b128_few_kernel<FA, FB, 4, 2, 8, OUT_BF16>
                                    : gemm_f8_b128_few_kernel<FA, FB, 4, 2, 4, OUT_BF16>;
            hipLaunchKernelGGL(kernel, dim3((unsigned)tiles), dim3(wide ? 512 : 256), 0, stream, a.M, a.N,
                               (int)(K_pad / 128), (int)tiles_n, a.A, a.As, a.B, a.Bs, a.bias, a.C, a.ldc);
            break;
        }
        case F8Form::kTiles128: {
            const int tiles_m = (int)cdiv(a.M, 128), tiles_n = (int)cdiv(a.N, 128);
            auto kernel = gemm_f8_b128_kernel<F8Small, FA, FB, OUT_BF16>;
            hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles_m * tiles_n)), dim3(F8Small::kThreads), 0, stream, a.M,
                               a.N, K_pad, tiles_m, tiles_n, kBandRows, a.A, a.As, a.B, a.Bs, a.bias, a.C, a.ldc);
            break;
        }
        case F8Form::kPersistent: {
            const int tiles_m = (int)cdiv(a.M, 256), tiles_n = (int)cdiv(a.N, 256), tiles = tiles_m * tiles_n;
            const int cus = device_cu_count();
            if constexpr (OUT_BF16)
                hipLaunchKernelGGL(a.bias ? (gemm_f8_b128_stream_kernel<F8Main, FA, FB, true>)
                                          : (gemm_f8_b128_stream_kernel<F8Main, FA, FB, false>),
                                   dim3((unsigned)(tiles < cus ? tiles : cus)), dim3(F8Main::kThreads), 0, stream,
                                   (int)a.M, (int)a.N, (int)K_pad, tiles_m, tiles_n, kBandRows, a.A, a.As, a.B, a.Bs,
                                   a.bias, a.C, (int)a.ldc);
            break;
        }
        case F8Form::kTiles256: {
            const int tiles_m = (int)cdiv(a.M, 256), tiles_n = (int)cdiv(a.N, 256);
            auto kernel = gemm_f8_b128_kernel<F8Main, FA, FB, OUT_BF16>;
            hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles_m * tiles_n)), dim3(F8Main::kThreads), 0, stream, a.M,
                               a.N, K_pad, tiles_m, tiles_n, kBandRows, a.A, a.As, a.B, a.Bs, a.bias, a.C,
                               a.ldc);
            break;
        }
    }
    return hipGetLastError();
}

template <int FA, int FB>
hipError_t launch_out(const F8GemmArgs &a, hipStream_t stream) {
    return a.out_dtype == MX_BF16 ? launch_formats<FA, FB, true>(a, stream) : launch_formats<FA, FB, false>(a, stream);
}

}  // namespace

hipError_t launch_gemm_f8_b128(const F8GemmArgs &a, hipStream_t stream) {
    if (a.K == 0) {
        const int64_t blocks = cdiv(a.M * a.N, 256);
        const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
        if (a.out_dtype == MX_BF16)
            hipLaunchKernelGGL(f8_fill_kernel<uint16_t>, grid, dim3(256), 0, stream, static_cast<uint16_t *>(a.C), a.M,
                               a.N, a.ldc, a.bias);
        else
            hipLaunchKernelGGL(f8_fill_kernel<float>, grid, dim3(256), 0, stream, static_cast<float *>(a.C), a.M, a.N,
                               a.ldc, a.bias);
        return hipGetLastError();
    }
    if (a.fmt_a == MX_FP8_E4M3)
        return a.fmt_b == MX_FP8_E4M3 ? launch_out<0, 0>(a, stream) : launch_out<0, 1>(a, stream);
    return a.fmt_b == MX_FP8_E4M3 ? launch_out<1, 0>(a, stream) : launch_out<1, 1>(a, stream);
}

hipError_t launch_linear_f8_b128(const F8LinearArgs &a, hipStream_t stream) {
    if (a.g.K > 0 && f8_linear_fused(a.g.M)) {
        if (a.g.fmt_a == MX_FP8_E4M3)
            return a.g.fmt_b == MX_FP8_E4M3 ? launch_linear<0, 0>(a, stream) : launch_linear<0, 1>(a, stream);
        return a.g.fmt_b == MX_FP8_E4M3 ? launch_linear<1, 0>(a, stream) : launch_linear<1, 1>(a, stream);
    }
    if (a.g.K > 0) {
        // (the workspace is the blob of x)
        const F8QuantArgs q{a.x, a.g.M, a.g.K, a.ldx, a.g.fmt_a, 0, false, false, const_cast<uint8_t *>(a.g.A),
                            const_cast<uint8_t *>(a.g.As), nullptr, nullptr};
        const hipError_t e = launch_quantize_f8_b128(q, MX_LAYOUT_TILED, stream);
        if (e != hipSuccess) return e;
    }
    return launch_gemm_f8_b128(a.g, stream);
}

}  // namespace mx
