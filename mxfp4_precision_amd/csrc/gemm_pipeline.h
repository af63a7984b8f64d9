// The software pipeline of the block-scaled GEMMs: element formats, tile
// shapes, LDS stages, the k-loop and the epilogues, shared by the kernels of
// gemm.hip (which describes it) and gemm_grouped.hip.
#pragma once

#include <type_traits>

#include "mx_internal.h"

namespace mx {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef uint32_t v6u __attribute__((ext_vector_type(6)));   // one lane's FP6 operand
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t v4u_t __attribute__((ext_vector_type(4)));
typedef uint32_t v2u_t __attribute__((ext_vector_type(2)));

// Offset that lies past every operand buffer: a buffer load there returns 0.
constexpr uint32_t kOutOfRange = 0x80000000u;
// buffer-store cache policy: non-temporal (C is not read again by the kernel)
constexpr int kCachePolicyNT = 2;
// s_waitcnt immediate for vmcnt(0) with expcnt and lgkmcnt left at their
// maxima (no wait): vmcnt bits [3:0] and [15:14], expcnt [6:4], lgkmcnt [11:8]
constexpr int kWaitVmcnt0 = 0x0F70;

// Buffer resource over [p, p + bytes).  Loads address it with a per-lane
// byte offset; an offset at or past `bytes` reads zeros (the hardware range
// check of raw buffers), which is how k-steps past K_pad become zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
}

#define MX_LDS(p) ((__attribute__((address_space(3))) void *)(p))

// ------------------------------------------------------------ element formats
// MFMA f8f6f4 format codes: 2 = E2M3, 3 = E3M2, 4 = E2M1.
struct Fp4Fmt {
    static constexpr int kFa = 4, kFb = 4;    // formats of A and B
    static constexpr bool kHi = false;        // an operand is one 16-byte slice
    static constexpr int kStepBytes = 1024;   // blob bytes of one 16-row group per k-step
    static constexpr int kStages = 4;
    static constexpr int kPeriod = 4;
    // the next k-group's scales go to a spare register set during the
    // group's last step (12 VGPRs that the FP4 operands leave room for)
    static constexpr bool kScaleAhead = true;
    // a separate copy of the k-loop for the steps whose DMAs all fall inside
    // the tile's K, without range tests (see dma_op)
    static constexpr bool kInner = true;
    static constexpr bool kStream = true;   // persistent form for bf16 output
    typedef uint4 Op;
};
template <int FA, int FB>
struct Fp6Fmt {
    static constexpr int kFa = FA, kFb = FB;
    static constexpr bool kHi = true;         // 16 bytes in the atom's first KB + 8 in its high part
    static constexpr int kStepBytes = 1536;
    static constexpr int kStages = 3;
    static constexpr int kPeriod = 12;
    // each half's scale entries are replaced while that half's MFMAs are not
    // running (the 6-register operands leave no room for a second set)
    static constexpr bool kScaleAhead = false;
    // one copy of the 12-step loop body: a second one costs spills
    static constexpr bool kInner = false;
    // The persistent form with its stores written straight from registers
    // (no stage is free for staging) measured 1.3-2.7x slower than one tile
    // per workgroup on the fc2 shapes: each 8-byte store instruction touches
    // 32 rows.
    static constexpr bool kStream = false;
    typedef v6u Op;
};

// ------------------------------------------------------------ tile shapes
// BM x BN workgroup tile of C, WM x WN wave tile, KG K groups (1, or 2 for
// the split form: waves [0, W) run the first half of K, [W, 2W) the second).
template <int BM, int BN, int WM, int WN, int KG>
struct Shape {
    static constexpr int kBM = BM, kBN = BN, kWM = WM, kWN = WN, kKG = KG;
    static constexpr int kWavesM = BM / WM;               // wave grid kWavesM x (BN / WN)
    static constexpr int kWaves = (BM / WM) * (BN / WN);  // waves of one K group
    static constexpr int kThreads = kWaves * KG * 64;
};
using MainShape = Shape<256, 256, 128, 64, 1>;
using TailShape = Shape<128, 128, 64, 64, 1>;
using SplitShape = Shape<128, 128, 64, 64, 2>;

template <class F, class S>
struct Cfg {
    using Fmt = F;
    using Op = typename F::Op;
    static constexpr int kStages = F::kStages, kPeriod = F::kPeriod;
    static constexpr int kBM = S::kBM, kBN = S::kBN, kWM = S::kWM, kWN = S::kWN, kKG = S::kKG;
    static constexpr int kWaves = S::kWaves, kWavesM = S::kWavesM, kThreads = S::kThreads;
    static constexpr int kGA = kBM / 16, kGB = kBN / 16;  // A / B atoms (16-row groups) per k-step
    static constexpr int kAtoms = kGA + kGB;
    static constexpr int kTA = kWM / 16, kTB = kWN / 16;  // atoms per wave tile
    static constexpr int kMA = kWM / 32, kMB = kWN / 32;  // 32x32 MFMA tiles per wave along M (A) / N (B)
    static constexpr int kSlots = kMA * kMB;              // MFMAs per wave per half-step
    // DMA units per wave and k-step: one 1 KB unit per atom (FP4: the atom;
    // FP6: its first KB), and for FP6 one per two atoms holding both high
    // parts, interleaved in 16-byte chunks (chunk c of atom 2h+a at position
    // 2c+a); scale atoms, 256 bytes each, when a step opens a k-group
    static constexpr int kLoLoads = kAtoms / kWaves;
    static constexpr int kHiLoads = F::kHi ? kAtoms / 2 / kWaves : 0;
    static constexpr int kLoads = kLoLoads + kHiLoads;
    static constexpr int kScaleLoads = kAtoms / kWaves;
    static constexpr int kHalfLoads = kLoads / 2, kHalfScale = kScaleLoads / 2;
    static constexpr int kHiBase = kAtoms * 1024;         // high-part units follow the first KBs
    static constexpr int kStageBytes = kAtoms * (F::kHi ? 1536 : 1024);
    static_assert(kAtoms % kWaves == 0 && kLoads % 2 == 0 && kScaleLoads % 2 == 0, "DMA split");
    static_assert(!F::kHi || kAtoms % (2 * kWaves) == 0, "whole high-part units per wave");
    static_assert(kMA + kMB <= kSlots, "one operand read per slot");

    // A k-step's DMA is issued in two parts: part P holds data units
    // [P*kHalfLoads, (P+1)*kHalfLoads) and, when the step opens a k-group
    // (k-group position SG == 0), scale units [P*kHalfScale, (P+1)*kHalfScale).
    static constexpr int part_ops(int SG) { return SG == 0 ? kHalfLoads + kHalfScale : kHalfLoads; }
    static constexpr int part_op(int P, int n) {
        return n < kHalfLoads ? kHalfLoads * P + n : kLoads + kHalfScale * P + (n - kHalfLoads);
    }
    // vector-memory instructions a wave issues for a k-step at k-group position SG
    static constexpr int issued_for(int SG) { return 2 * part_ops(SG); }
    // slot of the n-th of nv DMA instructions in a half-step
    static constexpr int dma_slot(int n, int nv) {
        const int s = 1 + (n * kSlots) / nv;
        return s > kSlots - 1 ? kSlots - 1 : s;
    }
    static_assert(part_ops(0) <= 5, "dma slots");
};

// LDS.  Each stage (and the scale k-group) is an array of its own, so that
// the compiler can tell a DMA into one stage from a read of another; K group
// G of the split form has its own set.
// ID: stage index (0..3) or 4 for the scale k-group, plus 8 per K group.
template <int BYTES, int ID>
__shared__ __attribute__((aligned(1024))) uint8_t g_lds[BYTES];
template <class C, int S, int G>
__device__ __forceinline__ uint8_t *stage_buf() {
    return g_lds<C::kStageBytes, 8 * G + S>;
}
template <class C, int G>
__device__ __forceinline__ uint8_t *scale_buf() {
    return g_lds<C::kAtoms * 256, 8 * G + 4>;
}
template <class C, int G = 0>
__device__ __forceinline__ uint8_t *stage_dyn(int s) {
    if constexpr (C::kStages == 4)
        return s == 0 ? stage_buf<C, 0, G>() : s == 1 ? stage_buf<C, 1, G>() : s == 2 ? stage_buf<C, 2, G>()
                                                                                     : stage_buf<C, 3, G>();
    else
        return s == 0 ? stage_buf<C, 0, G>() : s == 1 ? stage_buf<C, 1, G>() : stage_buf<C, 2, G>();
}

// After the k-loop the stages hold the bf16 C tile: kCRows rows per stage,
// kBN * 2 bytes per row, 16-byte chunk c of row r at chunk c ^ (r % chunks
// per row), so that reads and writes of a column of rows spread over all
// banks.  Byte address of bf16 element (r, col), col % 4 == 0.
template <class C>
__device__ __forceinline__ uint8_t *c_stage(int r, int col) {
    constexpr int kCRows = C::kStageBytes / (C::kBN * 2);
    constexpr int kChunks = C::kBN * 2 / 16;
    static_assert(kCRows * C::kStages >= C::kBM, "the bf16 C tile fits the stages");
    const int s = r / kCRows, rr = r - s * kCRows;
    const int chunk = (col >> 3) ^ (r & (kChunks - 1));
    return stage_dyn<C>(s) + rr * (C::kBN * 2) + chunk * 16 + (col & 7) * 2;
}

// ------------------------------------------------------------ pipeline state
// STREAM: the workgroup runs several output tiles back to back as one stream
// of k-steps; a tile occupies kstream steps of it, and a DMA for step kstream
// + j (j < 3) fetches step j of the next tile (*_next; knext = its k-steps, 0
// when there is none).
template <class C, bool STREAM>
struct Ctx {
    static constexpr bool kStream = STREAM;
    // k-step counter type: the stream kernel keeps k-steps in 32 bits (operand
    // blobs stay below 2 GiB, so K_pad / 128 < 2^24) to spare scalar registers
    using kint = typename std::conditional<STREAM, int, int64_t>::type;
    __amdgpu_buffer_rsrc_t rA, rB, rAs, rBs;
    int lo_row[C::kLoLoads];      // byte offsets of this wave's unit rows at k-step 0 (wave-uniform)
    uint32_t hi_off[C::kHiLoads > 0 ? C::kHiLoads : 1];   // FP6 high-part units: per lane, lane part included
    int sc_row[C::kScaleLoads];   // byte offsets of this wave's scale-atom rows at k-group 0
    kint ksteps, kgroups;
    int wave, lane16, lane4;
    int lo_next[STREAM ? C::kLoLoads : 1];
    uint32_t hi_next[STREAM && C::kHiLoads > 0 ? C::kHiLoads : 1];
    int sc_next[STREAM ? C::kScaleLoads : 1];
    kint kstream, knext;
};

template <class C>
struct Regs {
    using Op = typename C::Op;
    static constexpr bool kAhead = C::Fmt::kScaleAhead;
    Op a0[C::kMA], b0[C::kMB], a1[C::kMA], b1[C::kMB];   // operands of half 0 / half 1
    uint32_t sa[C::kMA][2], sb[C::kMB][2];                // scales of the k-group in use, per half
    uint32_t sa_n[kAhead ? C::kMA : 1][2], sb_n[kAhead ? C::kMB : 1][2];   // ... of the next one
};

// Per-lane LDS byte offsets of this wave's first A and B operand tiles (half
// 0), with the wave-dependent part folded in, so every read adds only a
// compile-time constant (tile, half) that fits the instruction's offset field.
struct Lds {
    int lo_a, lo_b;   // 16 bytes in a stage's first-KB region
    int hi_a, hi_b;   // FP6: 8 bytes in the interleaved high-part units
    int sc_a, sc_b;   // scale dword in the scale atoms
};

template <class C>
__device__ __forceinline__ Lds lds_offsets(int wave, int lane) {
    // lane L of a 32-row tile: row L%32 = atom (L%32)/16, slice s = L%16 + 16*(L/32) (half 0)
    const int wm = wave % C::kWavesM, wn = wave / C::kWavesM;
    const int lrow = lane & 31, lhi = lane >> 5;
    const int sl = (lrow & 15) + 16 * lhi;
    const int frag_off = ((lrow >> 4) * 1024) + sl * 16;
    // high parts: slice s of atom 2t + a at chunk position 2(s/2) + a, 8 bytes in per s%2
    const int frag_hi = 32 * (sl >> 1) + 16 * (lrow >> 4) + 8 * (sl & 1);
    // the slice's scale is byte (k-step % 4) of the dword at the same slice of the scale atom
    const int sc_off = ((lrow >> 4) * 256) + sl * 4;
    const int a0 = wm * C::kTA, b0 = C::kGA + wn * C::kTB;   // first atoms of the wave's A and B tiles
    Lds l;
    l.lo_a = frag_off + a0 * 1024;
    l.lo_b = frag_off + b0 * 1024;
    l.hi_a = frag_hi + (a0 / 2) * 1024;
    l.hi_b = frag_hi + (b0 / 2) * 1024;
    l.sc_a = sc_off + a0 * 256;
    l.sc_b = sc_off + b0 * 256;
    // Hide the bases' known zero bits: otherwise the compiler turns base +
    // constant into an OR, which the LDS instructions' offset field does not
    // take, and gives every read an address register of its own.
    asm volatile("" : "+v"(l.lo_a), "+v"(l.lo_b), "+v"(l.sc_a), "+v"(l.sc_b));
    if constexpr (C::Fmt::kHi) asm volatile("" : "+v"(l.hi_a), "+v"(l.hi_b));
    return l;
}

// Operand of one 32-row tile: 16 bytes from the first-KB region (plus 8 from
// the high part for FP6).
template <class C>
__device__ __forceinline__ typename C::Op read_op(const uint8_t *lo, const uint8_t *hi) {
    const uint4 v = *reinterpret_cast<const uint4 *>(lo);
    if constexpr (C::Fmt::kHi) {
        const uint2 h = *reinterpret_cast<const uint2 *>(hi);
        return v6u{v.x, v.y, v.z, v.w, h.x, h.y};
    } else {
        return v;
    }
}

// ZERO: the tile's first MFMA on these accumulators, which start from 0 (an
// inline constant, so the accumulators need no clearing between tiles).
template <class C, int SG, bool ZERO = false>
__device__ __forceinline__ void mfma_tile(v16f &acc, const typename C::Op &xb, const typename C::Op &xa, uint32_t sbv,
                                          uint32_t sav) {
    v8i bop, aop;
    if constexpr (C::Fmt::kHi) {
        bop = v8i{(int)xb[0], (int)xb[1], (int)xb[2], (int)xb[3], (int)xb[4], (int)xb[5], 0, 0};
        aop = v8i{(int)xa[0], (int)xa[1], (int)xa[2], (int)xa[3], (int)xa[4], (int)xa[5], 0, 0};
    } else {
        bop = v8i{(int)xb.x, (int)xb.y, (int)xb.z, (int)xb.w, 0, 0, 0, 0};
        aop = v8i{(int)xa.x, (int)xa.y, (int)xa.z, (int)xa.w, 0, 0, 0, 0};
    }
    // MFMA "A" operand = B rows (columns of C), "B" operand = A rows (rows of C);
    // OPSEL SG picks the k-step's byte of each scale dword
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bop, aop, ZERO ? v16f{} : acc, C::Fmt::kFb, C::Fmt::kFa, SG,
                                                          (int)sbv, SG, (int)sav);
}

// DMA instruction V of k-step k into stage S of K group G: V < kLoLoads
// copies the first KB of atom kWaves*V + wave; V < kLoads (FP6) the high
// parts of atoms 2h, 2h+1 (h = kWaves*(V - kLoLoads) + wave; lane p fetches
// chunk p/2 of atom 2h + p%2); otherwise (only when k opens a k-group) scale
// atom kWaves*(V - kLoads) + wave.  Past the operand's K the offset is out
// of range and the unit lands as zeros.  INNER: the caller guarantees k <
// ksteps (a step of the current tile inside K), so the offset is the row's
// plus k's with no test: a wave issues its instructions in order, and the
// tests and selects in front of every DMA otherwise hold back its next MFMA.
template <class C, int S, int V, int G, bool INNER, class X>
__device__ __forceinline__ void dma_op(const X &c, typename X::kint k) {
    using kint = typename X::kint;
    constexpr uint32_t kStep = C::Fmt::kStepBytes;
    if constexpr (V < C::kLoLoads) {
        // unit kWaves*V + wave: an A atom for every wave or a B atom for every wave
        constexpr bool isA = C::kWaves * (V + 1) <= C::kGA;
        static_assert(isA || C::kWaves * V >= C::kGA, "A/B split falls on a DMA instruction");
        const int a = C::kWaves * V + c.wave;
        const __amdgpu_buffer_rsrc_t rsrc = isA ? c.rA : c.rB;
        if constexpr (INNER) {
            // in range by construction: the wave-uniform part as the scalar
            // offset, the lane's constant part as the vector offset, so the
            // DMA needs no vector instruction of its own
            const uint32_t sbase = (uint32_t)c.lo_row[V] + (uint32_t)k * kStep;
            const uint32_t voff = (uint32_t)c.lane16;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, MX_LDS((stage_buf<C, S, G>() + a * 1024)), 16, voff, sbase,
                                                     0, 0);
            return;
        }
        uint32_t base;
        if constexpr (X::kStream) {
            // steps of the tile, then the next tile's first steps
            const bool cur = k < c.kstream;
            const kint kk = cur ? k : k - c.kstream;
            const int row = cur ? c.lo_row[V] : c.lo_next[V];
            base = kk < (cur ? c.ksteps : c.knext) ? (uint32_t)row + (uint32_t)kk * kStep : kOutOfRange;
        } else {
            base = k < c.ksteps ? (uint32_t)c.lo_row[V] + (uint32_t)k * kStep : kOutOfRange;
        }
        // (plain-typed locals: a builtin call on template-dependent operands
        // does not resolve in the host compilation pass)
        const uint32_t off = base + (uint32_t)c.lane16;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, MX_LDS((stage_buf<C, S, G>() + a * 1024)), 16, off, 0, 0, 0);
    } else if constexpr (V < C::kLoads) {
        constexpr int R = V - C::kLoLoads;
        constexpr bool isA = 2 * C::kWaves * (R + 1) <= C::kGA;
        static_assert(isA || 2 * C::kWaves * R >= C::kGA, "A/B split falls on a DMA instruction");
        const int h = C::kWaves * R + c.wave;
        uint32_t off;
        if constexpr (INNER) {
            off = c.hi_off[R] + (uint32_t)k * kStep;
        } else if constexpr (X::kStream) {
            const bool cur = k < c.kstream;
            const kint kk = cur ? k : k - c.kstream;
            const uint32_t row = cur ? c.hi_off[R] : c.hi_next[R];
            off = kk < (cur ? c.ksteps : c.knext) ? row + (uint32_t)kk * kStep : kOutOfRange;
        } else {
            off = k < c.ksteps ? c.hi_off[R] + (uint32_t)k * kStep : kOutOfRange;
        }
        const __amdgpu_buffer_rsrc_t rsrc = isA ? c.rA : c.rB;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, MX_LDS((stage_buf<C, S, G>() + C::kHiBase + h * 1024)), 16,
                                                 off, 0, 0, 0);
    } else {
        constexpr int R = V - C::kLoads;
        constexpr bool isA = C::kWaves * (R + 1) <= C::kGA;
        static_assert(isA || C::kWaves * R >= C::kGA, "A/B split falls on a DMA instruction");
        const int a = C::kWaves * R + c.wave;
        const kint h = k / 4;
        const __amdgpu_buffer_rsrc_t rsrc = isA ? c.rAs : c.rBs;
        if constexpr (INNER) {
            const uint32_t sbase = (uint32_t)c.sc_row[R] + (uint32_t)(h * 256);
            const uint32_t voff = (uint32_t)c.lane4;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, MX_LDS((scale_buf<C, G>() + a * 256)), 4, voff, sbase, 0, 0);
            return;
        }
        uint32_t base;
        {
            base = h < c.kgroups ? (uint32_t)c.sc_row[R] + (uint32_t)(h * 256) : kOutOfRange;
            // only step kstream (the next tile's first) opens a k-group past the tile
            if constexpr (X::kStream)
                if (k >= c.kstream) base = c.knext > 0 ? (uint32_t)c.sc_next[R] : kOutOfRange;
        }
        const uint32_t off = base + (uint32_t)c.lane4;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, MX_LDS((scale_buf<C, G>() + a * 256)), 4, off, 0, 0, 0);
    }
}

// Part P of the DMA of k-step k (stage S, k-group position SG).
template <class C, int S, int SG, int P, int G, int n = 0, class X>
__device__ __forceinline__ void dma_part(const X &c, typename X::kint k) {
    if constexpr (n < C::part_ops(SG)) {
        dma_op<C, S, C::part_op(P, n), G, false>(c, k);
        dma_part<C, S, SG, P, G, n + 1>(c, k);
    }
}

// Slot T of half H of the k-step with stage S and k-group position SG.
//  - MFMA T: tile (i, j) = (T / kMA, T % kMA) with the operands of half H.
//  - LDS read T (T < kMA + kMB) of the other operand set: half 0 reads the
//    second half of stage S, half 1 the first half of stage S+1, in order of
//    first use (b[0], a[0..kMA), b[1..kMB)).
//  - scales: kScaleAhead: at SG == 3, half 1 reads the next k-group's
//    scales, two per slot, into the spare set; otherwise half 1 at SG == 3
//    and half 0 at SG == 0 replace the entries of the half whose MFMAs are
//    not running (the scale atoms stay in LDS until step 1 of the group
//    issues the next group's DMA).
//  - the DMA instructions this slot carries (half 0: part 1 of step k+2,
//    half 1: part 0 of step k+3).  FRESH (a tile's first k-step in the
//    stream kernel): the second part of step 2 already went out before the
//    previous tile's stores.  INNER: both steps lie inside the tile's K.
template <class C, int S, int SG, int H, int T, bool FRESH, bool INNER, int G, class X>
__device__ __forceinline__ void slot(const X &c, typename X::kint k, v16f (&acc)[C::kMB][C::kMA], Regs<C> &r,
                                     const Lds &l) {
    constexpr int i = T / C::kMA, j = T % C::kMA;
    // a tile's first half-step in the stream kernel holds the first MFMA on every accumulator tile
    if constexpr (H == 0) mfma_tile<C, SG, FRESH && SG == 0>(acc[i][j], r.b0[i], r.a0[j], r.sb[i][0], r.sa[j][0]);
    else mfma_tile<C, SG>(acc[i][j], r.b1[i], r.a1[j], r.sb[i][1], r.sa[j][1]);

    if constexpr (T < C::kMA + C::kMB) {
        constexpr int RS = H == 0 ? S : (S + 1) % C::kStages;
        constexpr int RH = H == 0 ? 1 : 0;
        const uint8_t *st = stage_buf<C, RS, G>();
        if constexpr (T == 0 || T > C::kMA) {
            constexpr int bi = T == 0 ? 0 : T - C::kMA;
            const typename C::Op v = read_op<C>(st + l.lo_b + (2 * bi * 1024 + RH * 512),
                                                st + C::kHiBase + l.hi_b + (bi * 1024 + RH * 512));
            if constexpr (H == 0) r.b1[bi] = v; else r.b0[bi] = v;
        } else {
            constexpr int ai = T - 1;
            const typename C::Op v = read_op<C>(st + l.lo_a + (2 * ai * 1024 + RH * 512),
                                                st + C::kHiBase + l.hi_a + (ai * 1024 + RH * 512));
            if constexpr (H == 0) r.a1[ai] = v; else r.a0[ai] = v;
        }
    }
    constexpr int kScStart = C::kSlots - (C::kMA + C::kMB);
    const uint8_t *scb = scale_buf<C, G>();
    if constexpr (C::Fmt::kScaleAhead) {
        if constexpr (H == 1 && SG == 3 && T >= kScStart) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int q = 2 * (T - kScStart) + e;
                const int hh = q & 1, t = q >> 1;
                if (t < C::kMA)
                    r.sa_n[t][hh] = *reinterpret_cast<const uint32_t *>(scb + l.sc_a + 2 * t * 256 + hh * 128);
                else
                    r.sb_n[t - C::kMA][hh] =
                        *reinterpret_cast<const uint32_t *>(scb + l.sc_b + 2 * (t - C::kMA) * 256 + hh * 128);
            }
        }
    } else if constexpr (((H == 1 && SG == 3) || (H == 0 && SG == 0)) && T >= kScStart) {
        constexpr int t = T - kScStart, hh = 1 - H;   // the half whose MFMAs are not running
        if constexpr (t < C::kMA)
            r.sa[t][hh] = *reinterpret_cast<const uint32_t *>(scb + l.sc_a + (2 * t * 256 + hh * 128));
        else
            r.sb[t - C::kMA][hh] =
                *reinterpret_cast<const uint32_t *>(scb + l.sc_b + (2 * (t - C::kMA) * 256 + hh * 128));
    }

    constexpr int DS = H == 0 ? (S + 2) % C::kStages : (S + 3) % C::kStages;
    constexpr int DG = H == 0 ? (SG + 2) % 4 : (SG + 3) % 4;
    constexpr int P = H == 0 ? 1 : 0;
    constexpr int nv = (FRESH && SG == 0 && H == 0) ? 0 : C::part_ops(DG);
    const typename X::kint dk = H == 0 ? k + 2 : k + 3;
    if constexpr (nv > 0 && C::dma_slot(0, nv) == T) dma_op<C, DS, C::part_op(P, 0), G, INNER>(c, dk);
    if constexpr (nv > 1 && C::dma_slot(1, nv) == T) dma_op<C, DS, C::part_op(P, 1), G, INNER>(c, dk);
    if constexpr (nv > 2 && C::dma_slot(2, nv) == T) dma_op<C, DS, C::part_op(P, 2), G, INNER>(c, dk);
    if constexpr (nv > 3 && C::dma_slot(3, nv) == T) dma_op<C, DS, C::part_op(P, 3), G, INNER>(c, dk);
    if constexpr (nv > 4 && C::dma_slot(4, nv) == T) dma_op<C, DS, C::part_op(P, 4), G, INNER>(c, dk);
    // keep this slot's instructions in this slot
    __builtin_amdgcn_sched_barrier(0);
}

template <class C, int S, int SG, int H, bool FRESH, bool INNER, int G, int T = 0, class X>
__device__ __forceinline__ void half_step(const X &c, typename X::kint k, v16f (&acc)[C::kMB][C::kMA], Regs<C> &r,
                                          const Lds &l) {
    if constexpr (T < C::kSlots) {
        slot<C, S, SG, H, T, FRESH, INNER, G>(c, k, acc, r, l);
        half_step<C, S, SG, H, FRESH, INNER, G, T + 1>(c, k, acc, r, l);
    }
}

// One 128-wide k-step.  The barrier waits for this wave's DMA of step k+1
// (only step k+2's instructions may still be outstanding) and then for every
// wave, which publishes step k+1 and certifies that every read of the stage
// that half 1 starts overwriting is done.  Vector memory instructions
// complete in issue order (loads and stores alike), so the count is exact.
// FRESH: the first k-steps of a tile in the stream kernel, where EXTRA
// vector-memory instructions (the previous tile's stores and this tile's
// bias loads) were issued after all of step 2's DMA; the first two waits
// count past them instead of draining them.
template <class C, int S, int SG, bool FRESH, int EXTRA, bool INNER, int G, class X>
__device__ __forceinline__ void k_step(const X &c, typename X::kint k, v16f (&acc)[C::kMB][C::kMA], Regs<C> &r,
                                       const Lds &l) {
    constexpr int kStores = FRESH && SG < 2 ? EXTRA : 0;
    // with a 12-step loop body an opaque step index keeps the compiler from
    // precomputing every step's addresses into registers
    if constexpr (C::kPeriod > 4) asm volatile("" : "+s"(k));
    __builtin_amdgcn_sched_barrier(0);
    half_step<C, S, SG, 0, FRESH, INNER, G>(c, k, acc, r, l);
    static_assert(C::issued_for((SG + 2) & 3) + kStores <= 63, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(C::issued_for((SG + 2) & 3) + kStores) : "memory");
    __builtin_amdgcn_sched_barrier(0);
    half_step<C, S, SG, 1, FRESH, INNER, G>(c, k, acc, r, l);
    if constexpr (C::Fmt::kScaleAhead && SG == 3) {
#pragma unroll
        for (int t = 0; t < C::kMA; ++t) { r.sa[t][0] = r.sa_n[t][0]; r.sa[t][1] = r.sa_n[t][1]; }
#pragma unroll
        for (int t = 0; t < C::kMB; ++t) { r.sb[t][0] = r.sb_n[t][0]; r.sb[t][1] = r.sb_n[t][1]; }
    }
}

// kPeriod consecutive k-steps from k0 (stage and k-group position 0 at k0).
// FRESH applies to the first two.
template <class C, bool FRESH, int EXTRA, bool INNER, int G, int s = 0, class X>
__device__ __forceinline__ void period(const X &c, typename X::kint k0, v16f (&acc)[C::kMB][C::kMA], Regs<C> &r,
                                       const Lds &l) {
    if constexpr (s < C::kPeriod) {
        k_step<C, s % C::kStages, s % 4, FRESH && s < 2, EXTRA, INNER, G>(c, k0 + s, acc, r, l);
        period<C, FRESH, EXTRA, INNER, G, s + 1>(c, k0, acc, r, l);
    }
}

// Scales of k-group 0 (both halves) and the operands of step 0's half 0,
// once the prologue's DMA has landed for every wave.
template <class C, int G>
__device__ __forceinline__ void first_operands(Regs<C> &r, const Lds &l) {
    const uint8_t *scb = scale_buf<C, G>();
    const uint8_t *st = stage_buf<C, 0, G>();
#pragma unroll
    for (int t = 0; t < C::kMA; ++t)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
            r.sa[t][hh] = *reinterpret_cast<const uint32_t *>(scb + l.sc_a + t * 512 + hh * 128);
#pragma unroll
    for (int t = 0; t < C::kMB; ++t)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
            r.sb[t][hh] = *reinterpret_cast<const uint32_t *>(scb + l.sc_b + t * 512 + hh * 128);
#pragma unroll
    for (int t = 0; t < C::kMA; ++t)
        r.a0[t] = read_op<C>(st + l.lo_a + t * 2048, st + C::kHiBase + l.hi_a + t * 1024);
#pragma unroll
    for (int t = 0; t < C::kMB; ++t)
        r.b0[t] = read_op<C>(st + l.lo_b + t * 2048, st + C::kHiBase + l.hi_b + t * 1024);
}

// ------------------------------------------------------------ tile order
// Position `id` of the tile order: bands of group_m tile rows, walked column
// by column.
__device__ __forceinline__ void tile_at(int id, int tiles_m, int tiles_n, int group_m, int &tm, int &tn) {
    const int band = group_m * tiles_n;
    const int first_m = (id / band) * group_m;
    const int gsz = min(tiles_m - first_m, group_m);
    tm = first_m + (id % band) % gsz;
    tn = (id % band) / gsz;
}

// Tile of block index b in a launch of nb blocks: XCD-contiguous ranges of
// the tile order (blocks are dispatched to the XCDs round-robin).
__device__ __forceinline__ void tile_of(int b, int nb, int tiles_m, int tiles_n, int group_m, int &tm, int &tn) {
    const int xcd = b % kXcds, local = b / kXcds;
    const int per = nb / kXcds, rem = nb % kXcds;
    tile_at(xcd * per + (xcd < rem ? xcd : rem) + local, tiles_m, tiles_n, group_m, tm, tn);
}

// Byte offsets of this wave's unit rows and scale-atom rows for tile (tm,
// tn), starting at k-step kfirst (a multiple of 4).  Row groups past an
// operand are clamped to its last group: those rows of C are never stored,
// so their contents do not matter.
template <class C, class X>
__device__ __forceinline__ void tile_rows(const X &c, int tm, int tn, int64_t nGA, int64_t nGB, int64_t ksteps,
                                          int64_t kgroups, int64_t kfirst, int lane, int (&lo)[C::kLoLoads],
                                          uint32_t (&hi)[C::kHiLoads > 0 ? C::kHiLoads : 1],
                                          int (&sc)[C::kScaleLoads]) {
    const int64_t gA0 = (int64_t)tm * C::kGA, gB0 = (int64_t)tn * C::kGB;
    auto group_of = [&](int a) -> int64_t {
        const bool isA = a < C::kGA;
        const int64_t g = isA ? gA0 + a : gB0 + (a - C::kGA);
        const int64_t gmax = (isA ? nGA : nGB) - 1;
        return g < gmax ? g : gmax;
    };
    constexpr int64_t kStep = C::Fmt::kStepBytes;
#pragma unroll
    for (int r = 0; r < C::kLoLoads; ++r)
        lo[r] = (int)((group_of(C::kWaves * r + c.wave) * ksteps + kfirst) * kStep);
    if constexpr (C::kHiLoads > 0) {
#pragma unroll
        for (int r = 0; r < C::kHiLoads; ++r) {
            const int h = C::kWaves * r + c.wave;
            hi[r] = (uint32_t)((group_of(2 * h + (lane & 1)) * ksteps + kfirst) * kStep) + 1024u +
                    (uint32_t)((lane >> 1) * 16);
        }
    }
#pragma unroll
    for (int r = 0; r < C::kScaleLoads; ++r)
        sc[r] = (int)((group_of(C::kWaves * r + c.wave) * kgroups + kfirst / 4) * 256);
}

// ------------------------------------------------------------ bias
// This lane's bias values for tile column tn: columns n0 + 32i + 8q +
// 4(lane/32) + 0..3 of its wave tile, 4 bf16 per (i, q), one 8-byte buffer
// load each, issued before the k-loop so they have long arrived by the
// epilogue.  The range check of a buffer load zeroes whole dwords, so the
// range ends at the 16-byte boundary after the last entry (the bias is
// 16-byte aligned, so that block is inside its allocation's last page);
// columns past it read 0, columns past N are never stored.
template <class C>
__device__ __forceinline__ void load_bias(__amdgpu_buffer_rsrc_t rb, int tn, int wn, int lane,
                                          v2u_t (&bias_bits)[C::kMB * 4]) {
    const int col0 = tn * C::kBN + wn * C::kWN + 4 * (lane >> 5);
#pragma unroll
    for (int i = 0; i < C::kMB; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            bias_bits[i * 4 + q] = __builtin_amdgcn_raw_buffer_load_b64(rb, (col0 + 32 * i + 8 * q) * 2, 0, 0);
}

// C[i][j] = (sum) + bias[j], added in fp32 before the output rounding.
template <class C>
__device__ __forceinline__ void add_bias(v16f (&acc)[C::kMB][C::kMA], const v2u_t (&bias_bits)[C::kMB * 4]) {
#pragma unroll
    for (int i = 0; i < C::kMB; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const v2u_t bb = bias_bits[i * 4 + q];
            const float b0 = __uint_as_float(bb[0] << 16), b1 = __uint_as_float(bb[0] & 0xFFFF0000u);
            const float b2 = __uint_as_float(bb[1] << 16), b3 = __uint_as_float(bb[1] & 0xFFFF0000u);
#pragma unroll
            for (int j = 0; j < C::kMA; ++j) {
                acc[i][j][4 * q] += b0;
                acc[i][j][4 * q + 1] += b1;
                acc[i][j][4 * q + 2] += b2;
                acc[i][j][4 * q + 3] += b3;
            }
        }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

// ------------------------------------------------------------ epilogues
// Write the tile (tm, tn) of C from the accumulators;
// acc[i][j][r] = C[m0 + 32j + lane%32][n0 + 32i + 8(r/4) + 4(lane/32) + r%4].
// bf16: rounded (V_CVT_PK_BF16_F32, nearest even), staged in LDS, then
// written as whole row segments (16 bytes per lane; non-temporal, as C is
// not read again here); fp32: 16 bytes per lane straight from registers.
// Masked at the M/N edges.  With two K groups, group 0 holds the summed
// accumulators (wave = its index in the group); all waves (index wave_all)
// take part in the bf16 stores.
template <class C, bool OUT_BF16>
__device__ __forceinline__ void store_tile(v16f (&acc)[C::kMB][C::kMA], int tm, int tn, int64_t M, int64_t N,
                                           void *Cout, int64_t ldc, int group, int wave, int wave_all, int lane) {
    const int wm = wave % C::kWavesM, wn = wave / C::kWavesM;
    const int lrow = lane & 31, lhi = lane >> 5;
    const int64_t tm0 = (int64_t)tm * C::kBM, tn0 = (int64_t)tn * C::kBN;
    if (OUT_BF16) {
        // Every wave waited for its own DMAs; the barrier makes sure all of
        // them have landed and every stage read is done before the tile
        // overwrites the stages.
        __syncthreads();
        if (group == 0) {
#pragma unroll
            for (int j = 0; j < C::kMA; ++j)
#pragma unroll
                for (int i = 0; i < C::kMB; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int rl = wm * C::kWM + 32 * j + lrow, cl = wn * C::kWN + 32 * i + 8 * q + 4 * lhi;
                        *reinterpret_cast<uint2 *>(c_stage<C>(rl, cl)) =
                            uint2{pack_bf16x2(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                                  pack_bf16x2(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3])};
                    }
        }
        __syncthreads();
        constexpr int kLanesPerRow = C::kBN * 2 / 16;        // 32 (256 columns) or 16 (128)
        constexpr int kRowsPerInst = 64 / kLanesPerRow;
        constexpr int kRowsPerWave = C::kBM / (C::kWaves * C::kKG);
        constexpr int kInst = kRowsPerWave / kRowsPerInst;
        const int cl = (lane % kLanesPerRow) * 8;
        const int64_t col = tn0 + cl;
        const int rsub = lane / kLanesPerRow;
        uint4 v[kInst];
#pragma unroll
        for (int it = 0; it < kInst; ++it)
            v[it] = *reinterpret_cast<const uint4 *>(c_stage<C>(kRowsPerWave * wave_all + kRowsPerInst * it + rsub, cl));
        uint16_t *dst0 = reinterpret_cast<uint16_t *>(Cout) + (tm0 + kRowsPerWave * wave_all + rsub) * ldc + col;
        if (tm0 + C::kBM <= M && tn0 + C::kBN <= N) {
#pragma unroll
            for (int it = 0; it < kInst; ++it)
                __builtin_nontemporal_store(__builtin_bit_cast(v4u_t, v[it]),
                                            reinterpret_cast<v4u_t *>(dst0 + kRowsPerInst * it * ldc));
        } else {
#pragma unroll
            for (int it = 0; it < kInst; ++it) {
                const int64_t row = tm0 + kRowsPerWave * wave_all + kRowsPerInst * it + rsub;
                if (row >= M || col >= N) continue;
                uint16_t *dst = dst0 + kRowsPerInst * it * ldc;
                if (col + 7 < N) {
                    *reinterpret_cast<uint4 *>(dst) = v[it];
                } else {
                    const uint32_t w4[4] = {v[it].x, v[it].y, v[it].z, v[it].w};
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (col + e < N) dst[e] = (uint16_t)(w4[e >> 1] >> (16 * (e & 1)));
                }
            }
        }
    } else {
        if (group != 0) return;
        const int64_t m0 = tm0 + wm * C::kWM, n0 = tn0 + wn * C::kWN;
#pragma unroll
        for (int j = 0; j < C::kMA; ++j) {
            const int64_t row = m0 + 32 * j + lrow;
            if (row >= M) continue;
#pragma unroll
            for (int i = 0; i < C::kMB; ++i) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t col = n0 + 32 * i + 8 * q + 4 * lhi;
                    const v4f v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                    float *dst = reinterpret_cast<float *>(Cout) + row * ldc + col;
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
    }
}

// Epilogue of the stream kernel (bf16 output, four stages).  Stages 0-2
// already hold the next tile's first k-steps, so only stage 3 is free.  Each
// wave takes a 4 KB slot of it: in pass p (kMA passes) the wave stages its own
// 32 x 64 block (MFMA row tile p: tile rows 128 wm + 32p + [0, 32), columns
// 64 wn + [0, 64)), 128 bytes per row with 16-byte chunk c of row r at c ^
// (r % 8), and reads it back as whole 128-byte row segments, 8 rows per store
// instruction.  After the first barrier (every wave done with stage 3's last
// k-step) no wave waits for another: a wave's LDS operations complete in
// order, so its next pass may overwrite the slot it has just read.  Every
// wave issues exactly epi_stores<C>() buffer stores per tile whatever the
// edges: a chunk past row M or column N gets an out-of-range offset, which
// the buffer range check drops (N % 8 == 0, so a chunk is all in or all out).
// The fixed count is what lets the next tile's first waits count past the
// stores instead of draining them.  Before the stores, the epilogue issues
// the second part of the next tile's step 2 (its first k-step would
// otherwise issue it after them), into stage 2, free since the tile's last
// k-step.  (Three stages would leave no stage free at a tile boundary, which
// is why the FP6 format has no persistent form.)
template <class C>
__host__ __device__ constexpr int epi_stores() {
    return C::kMA * 4;
}

// ODD: N need not be a multiple of 8, nor rows of C start on 128-byte lines.
// The chunk that N ends in is then written by elements, after its whole store
// was dropped (more stores than the fixed count only make the next tile's
// first waits longer), and no store is non-temporal, as neighbouring segments
// share lines.
template <class C, bool ODD = false>
__device__ __forceinline__ void store_tile_private(v16f (&acc)[C::kMB][C::kMA], int tm, int tn, int M, int N,
                                                   __amdgpu_buffer_rsrc_t rC, int ldc, int wave, int lane) {
    static_assert(C::kStages == 4, "the stream epilogue stages C through stage 3");
    constexpr int kSlotBytes = 32 * C::kWN * 2;   // 4 KB per wave
    static_assert(kSlotBytes * C::kWaves == C::kStageBytes, "one slot per wave fills stage 3");
    static_assert(C::kWN == 64, "8 lanes per 128-byte row");
    const int wm = wave % C::kWavesM, wn = wave / C::kWavesM;
    const int lrow = lane & 31, lhi = lane >> 5;
    const int row_w = tm * C::kBM + C::kWM * wm;                  // first C row of this wave's block
    const int col = tn * C::kBN + C::kWN * wn + 8 * (lane & 7);   // this lane's 8 columns on the way out
    uint8_t *slot_base = stage_buf<C, 3, 0>() + wave * kSlotBytes;
    auto c_slot = [&](int r, int chunk) { return slot_base + r * (C::kWN * 2) + ((chunk ^ (r & 7)) * 16); };
    // every wave is done reading stage 3 (the tile's last k-step); a bare
    // barrier: a __syncthreads() fence would also wait for the next tile's DMAs
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int p = 0; p < C::kMA; ++p) {
#pragma unroll
        for (int i = 0; i < C::kMB; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint2 *>(c_slot(lrow, 4 * i + q) + 8 * lhi) =
                    uint2{pack_bf16x2(acc[i][p][4 * q], acc[i][p][4 * q + 1]),
                          pack_bf16x2(acc[i][p][4 * q + 2], acc[i][p][4 * q + 3])};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = 8 * s + (lane >> 3);
            const v4u_t v = *reinterpret_cast<const v4u_t *>(c_slot(r, lane & 7));
            const int row = row_w + 32 * p + r;
            const bool in = row < M && col < N, whole = !ODD || col + 8 <= N;
            const uint32_t at = (uint32_t)(row * ldc + col) * 2u, off = in && whole ? at : kOutOfRange;
            __builtin_amdgcn_raw_buffer_store_b128(v, rC, off, 0, ODD ? 0 : kCachePolicyNT);
            if constexpr (ODD) {
                const int first = tn * C::kBN + C::kWN * wn;   // the wave's columns
                if (N % 8 != 0 && first < N && N < first + C::kWN) {
#pragma unroll
                    for (int e = 0; e < 7; ++e) {
                        if (e >= N % 8) break;
                        const short h = (short)(v[e >> 1] >> (16 * (e & 1)));
                        const uint32_t at_e = in && !whole && col + e < N ? at + 2u * e : kOutOfRange;
                        __builtin_amdgcn_raw_buffer_store_b16(h, rC, at_e, 0, 0);
                    }
                }
            }
        }
    }
}

template <class C>
__device__ __forceinline__ void store_tile_stream(const Ctx<C, true> &c, v16f (&acc)[C::kMB][C::kMA], int tm, int tn,
                                                  int M, int N, __amdgpu_buffer_rsrc_t rC, int ldc, int wave,
                                                  int lane) {
    dma_part<C, 2, 2, 1, 0>(c, c.kstream + 2);
    store_tile_private<C>(acc, tm, tn, M, N, rC, ldc, wave, lane);
}

// ------------------------------------------------------------ kernels
// The k-loop of K group G over `steps` k-steps (a multiple of 4; steps at or
// past c.ksteps land as zeros): prologue DMAs, whole periods, then the drain
// of the trailing DMAs.
template <class C, int G, class X>
__device__ __forceinline__ void run_tile(const X &c, v16f (&acc)[C::kMB][C::kMA], const Lds &l, int64_t steps) {
    // Prologue: steps 0 and 1 whole, the first part of step 2 (its second
    // part goes out in step 0's first half).
    dma_part<C, 0, 0, 0, G>(c, 0);
    dma_part<C, 0, 0, 1, G>(c, 0);
    dma_part<C, 1, 1, 0, G>(c, 1);
    dma_part<C, 1, 1, 1, G>(c, 1);
    dma_part<C, 2, 2, 0, G>(c, 2);
    Regs<C> r;
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(C::issued_for(1) + C::part_ops(2)) : "memory");
    first_operands<C, G>(r, l);
    // a period from k0 fetches steps k0+2 .. k0+kPeriod+2: inside K while
    // k0 + kPeriod + 2 < ksteps
    int64_t k0 = 0;
    if constexpr (C::Fmt::kInner)
        for (; k0 < steps && k0 + C::kPeriod + 2 < c.ksteps; k0 += C::kPeriod)
            period<C, false, 0, true, G>(c, k0, acc, r, l);
    for (; k0 < steps; k0 += C::kPeriod) period<C, false, 0, false, G>(c, k0, acc, r, l);
    // drain the trailing (out-of-range) DMAs before LDS is reused
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Split form: 4 KB of the second group's stages per accumulator tile of a
// wave (block w * kSlots + t), float e of lane L at (e * 64 + L) * 4, so
// consecutive lanes touch consecutive banks.
template <class C>
__device__ __forceinline__ float *partial_slot(int wave, int tile) {
    constexpr int kPerStage = C::kStageBytes / 4096;
    static_assert(C::kStageBytes % 4096 == 0 && C::kWaves * C::kSlots <= kPerStage * C::kStages, "partials fit");
    const int b = wave * C::kSlots + tile;
    return reinterpret_cast<float *>(stage_dyn<C, 1>(b / kPerStage) + (b % kPerStage) * 4096);
}

}  // namespace
}  // namespace mx
