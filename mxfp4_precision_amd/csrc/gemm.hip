// Block-scaled GEMMs (C = A . B^T) for gfx950: one software pipeline for
// MXFP4 (E2M1) and MXFP6 (E2M3 / E3M2) operands in the tiled blob layout,
// instantiated per element format and workgroup tile shape, plus the
// tensorwise-scaled FP8 (E5M2) product of the hybrid backward.
//
// C[i][j] = sum_k e(A[i][k]) 2^(sa[i][k/32]-127) * e(B[j][k]) 2^(sb[j][k/32]-127),
// fp32 accumulation, bf16 (RNE) or fp32 output: the NT product that the
// forward, dgrad and wgrad of the MXFP4 linear on the page
// "primus_turbo_mxfp4_local.py" compute (and its MXFP6 variant, with the
// element formats of OCP MX v1.0 sec. 5.3.2).
//
// MFMA: V_MFMA_SCALE_F32_32X32X64_F8F6F4.  Lane L of a 32-row operand tile
// supplies the 32 elements of row L%32, k-block 2*half + L/32 of a 128-wide
// k-step (16 bytes for FP4, 24 for FP6), and that block's E8M0 scale as the
// byte of a VGPR that OPSEL picks.  The tiled layout puts exactly those bytes
// at a fixed slice of an atom (16 rows x 128 k: 1 KB for FP4; 1536 bytes for
// FP6, each lane's first 16 bytes in the atom's first kilobyte and the last 8
// in the remaining 512 bytes) and a lane's scales for 4 consecutive k-steps
// in one dword of a 256-byte scale atom, so operands move as whole atoms and
// are read from LDS with conflict-free ds_read_b128 (plus ds_read_b64 for the
// FP6 high parts).
//
// Workgroup shapes: 256x256 tiles with 8 waves of 128x64 (4x2 MFMA tiles,
// 128 fp32 accumulators per lane, two waves per SIMD), and 128x128 tiles
// with 4 waves of 64x64 for the leftover tiles of a last round, alone or as
// two K groups of 4 waves that each run the pipeline over half of K and add
// their partial tiles through LDS.  Every LDS read or DMA instruction a wave
// issues stalls that wave's MFMA stream for tens of cycles; with two waves
// per SIMD the other wave's MFMAs fill that gap.
//
// Pipeline: LDS holds kStages k-step stages (FP4: 4 of 32 atoms, 32 KB each;
// FP6: 3 of 48 KB) and one k-group (4 steps) of scale atoms.  Atoms travel
// global -> LDS by DMA (buffer_load ... lds, no registers).  Each k-step is
// two halves of kSlots MFMAs per wave; one slot = one MFMA plus, in fixed
// order, the LDS read of an operand of the next half and the DMA
// instructions assigned to that slot, so memory instructions are spread
// evenly between MFMAs.  Half 0 of step k issues the second part of step
// k+2's DMA, half 1 the first part of step k+3's; the barrier between the
// halves publishes step k+1 and frees the stage that step k+3 lands in
// (step k-1's with four stages, step k's own with three).  The stage index
// runs mod kStages and the position in the 4-step scale group mod 4, so the
// unrolled k-loop body is kPeriod = lcm(kStages, 4) steps.
//
// The MFMA is issued with B as the "A" operand, so each lane's accumulators
// are 4 consecutive columns of one row of C.  Workgroups are ordered so that
// each XCD (8 on MI355X, dispatched round-robin) works on a compact band of
// output tiles, keeping the A rows and B columns it shares within its own L2.
//
// With a short K and several rounds of tiles, a persistent form runs one
// workgroup per CU over its tiles as one stream of k-steps: the next tile's
// first steps are fetched during the current tile's last ones, and the
// epilogue's stores drain while the next tile computes instead of holding
// the CU (at 24 k-steps per tile the bf16 stores alone cost ~10% otherwise).

#include <atomic>

#include "gemm_pipeline.h"

namespace mx {
namespace {

// One output tile per workgroup.  256x256 (the main order: workgroup b takes
// tile b of the XCD-remapped order) or 128x128 (the tail: workgroup b
// computes quarter b % 4 of 256x256 tile first + b / 4 of the main order).
// Two K groups (split form): group g = wave / 4 takes k-groups [g * kg0, ...)
// of the tile (kg0 = half of them, rounded up); group 1's partial tile is
// added into group 0's through LDS before the epilogue.  Every wave runs the
// same number of k-steps (group 1's past its K land as zeros), so the
// per-step barriers line up across groups.
// BIAS: C[i][j] = (sum) + bias[j], bias a bf16 vector of N.
template <class C, bool OUT_BF16, bool BIAS>
__global__ __launch_bounds__(C::kThreads) void gemm_kernel(int64_t M, int64_t N, int64_t K_pad, int tiles_m,
                                                           int tiles_n, int group_m, int first,
                                                           const uint8_t *__restrict__ A,
                                                           const uint8_t *__restrict__ As,
                                                           const uint8_t *__restrict__ B,
                                                           const uint8_t *__restrict__ Bs,
                                                           const uint16_t *__restrict__ bias, void *__restrict__ Cout,
                                                           int64_t ldc) {
    constexpr bool kSplit = C::kKG == 2;
    const int lane = threadIdx.x & 63;
    const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // wave-uniform
    const int group = kSplit ? wave_all / C::kWaves : 0;
    const int wave = wave_all % C::kWaves;
    const int wn = wave / C::kWavesM;

    int tm, tn;
    if constexpr (C::kBM == 256) {
        tile_of(blockIdx.x, gridDim.x, tiles_m, tiles_n, group_m, tm, tn);
    } else {
        const int quarter = (int)(blockIdx.x & 3);
        tile_at(first + (int)(blockIdx.x >> 2), tiles_m, tiles_n, group_m, tm, tn);
        tm = 2 * tm + (quarter >> 1);
        tn = 2 * tn + (quarter & 1);
    }

    const int64_t ksteps = K_pad / 128, kgroups = cdiv(K_pad, 512);
    // k-groups of group 0 (all of them without the split); group 1 starts at k-group kg0
    const int64_t kg0 = kSplit ? (kgroups + 1) / 2 : kgroups;
    const int64_t kfirst = group ? 4 * kg0 : 0;
    Ctx<C, false> c;
    c.ksteps = group ? ksteps - kfirst : (kSplit ? (ksteps < 4 * kg0 ? ksteps : 4 * kg0) : ksteps);
    c.kgroups = group ? kgroups - kg0 : kg0;
    c.wave = wave;
    c.lane16 = lane * 16;
    c.lane4 = lane * 4;
    const int64_t nGA = cdiv(M, 16), nGB = cdiv(N, 16);   // row groups present in memory
    constexpr int64_t kStep = C::Fmt::kStepBytes;
    c.rA = make_rsrc(A, nGA * ksteps * kStep);
    c.rB = make_rsrc(B, nGB * ksteps * kStep);
    c.rAs = make_rsrc(As, nGA * kgroups * 256);
    c.rBs = make_rsrc(Bs, nGB * kgroups * 256);

    v2u_t bias_bits[BIAS ? C::kMB * 4 : 1];
    if constexpr (BIAS) load_bias<C>(make_rsrc(bias, cdiv(N * 2, 16) * 16), tn, wn, lane, bias_bits);
    // a group's offsets start at its first k-step
    tile_rows<C>(c, tm, tn, nGA, nGB, ksteps, kgroups, kfirst, lane, c.lo_row, c.hi_off, c.sc_row);

    v16f acc[C::kMB][C::kMA];
#pragma unroll
    for (int i = 0; i < C::kMB; ++i)
#pragma unroll
        for (int j = 0; j < C::kMA; ++j) acc[i][j] = v16f{};

    const Lds l = lds_offsets<C>(wave, lane);
    const int64_t steps = 4 * kg0;   // k-steps every wave runs
    if (kSplit && group == 1) run_tile<C, 1>(c, acc, l, steps);
    else run_tile<C, 0>(c, acc, l, steps);

    if constexpr (kSplit) {
        // every wave is past its last stage read; group 1's stages take its partial tile
        __syncthreads();
        if (group == 1) {
#pragma unroll
            for (int i = 0; i < C::kMB; ++i)
#pragma unroll
                for (int j = 0; j < C::kMA; ++j) {
                    float *p = partial_slot<C>(wave, i * C::kMA + j) + lane;
#pragma unroll
                    for (int e = 0; e < 16; ++e) p[e * 64] = acc[i][j][e];
                }
        }
        __syncthreads();
        if (group == 0) {
#pragma unroll
            for (int i = 0; i < C::kMB; ++i)
#pragma unroll
                for (int j = 0; j < C::kMA; ++j) {
                    const float *p = partial_slot<C>(wave, i * C::kMA + j) + lane;
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][j][e] += p[e * 64];
                }
        }
    }
    if constexpr (BIAS)
        if (group == 0) add_bias<C>(acc, bias_bits);
    store_tile<C, OUT_BF16>(acc, tm, tn, M, N, Cout, ldc, group, wave, wave_all, lane);
}

// Persistent form of gemm_kernel (256x256 tiles, bf16 output): gridDim.x
// workgroups, block b runs tiles b, b + gridDim.x, ... of the first `tiles`
// of the tile order as one stream of k-steps.  A tile's last k-steps already
// fetch the next tile's first three and its first operands and scales, so
// the pipeline never drains between tiles; the epilogue's stores then
// overlap the next tile's first k-steps (its first two waits count past
// them, only the third one needs them done).  A tile is kstream = 4 *
// kgroups steps of the stream, a multiple of kPeriod, so every tile starts
// at stage 0.  BIAS: a tile's bias values are loaded right after the
// previous tile's stores (kMB * 4 more instructions for those waits to count
// past).  Needs N % 8 == 0 and M * ldc * 2 < 2^31 (32-bit store offsets).
template <class C, bool BIAS>
__global__ __launch_bounds__(C::kThreads) void gemm_stream_kernel(int M, int N, int K_pad, int tiles_m, int tiles_n,
                                                                  int group_m, int tiles,
                                                                  const uint8_t *__restrict__ A,
                                                                  const uint8_t *__restrict__ As,
                                                                  const uint8_t *__restrict__ B,
                                                                  const uint8_t *__restrict__ Bs,
                                                                  const uint16_t *__restrict__ bias,
                                                                  void *__restrict__ Cout, int ldc) {
    static_assert(C::kKG == 1 && C::kBM == 256, "stream form: main tiles");
    constexpr int kBiasLoads = BIAS ? C::kMB * 4 : 0;
    constexpr int kFreshOps = epi_stores<C>() + kBiasLoads;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave / C::kWavesM;
    const int P = gridDim.x;

    Ctx<C, true> c;
    c.ksteps = K_pad / 128;
    c.kgroups = (K_pad + 511) / 512;
    c.kstream = 4 * c.kgroups;
    c.wave = wave;
    c.lane16 = lane * 16;
    c.lane4 = lane * 4;
    const int nGA = (M + 15) / 16, nGB = (N + 15) / 16;
    constexpr int64_t kStep = C::Fmt::kStepBytes;
    c.rA = make_rsrc(A, (int64_t)nGA * c.ksteps * kStep);
    c.rB = make_rsrc(B, (int64_t)nGB * c.ksteps * kStep);
    c.rAs = make_rsrc(As, (int64_t)nGA * c.kgroups * 256);
    c.rBs = make_rsrc(Bs, (int64_t)nGB * c.kgroups * 256);
    const __amdgpu_buffer_rsrc_t rC = make_rsrc(Cout, (int64_t)M * ldc * 2);
    const __amdgpu_buffer_rsrc_t rBias = make_rsrc(bias, BIAS ? ((int64_t)N * 2 + 15) / 16 * 16 : 0);

    int vb = blockIdx.x;
    int tm, tn, tm_next = 0, tn_next = 0;
    tile_of(vb, tiles, tiles_m, tiles_n, group_m, tm, tn);
    tile_rows<C>(c, tm, tn, nGA, nGB, c.ksteps, c.kgroups, 0, lane, c.lo_row, c.hi_off, c.sc_row);
    c.knext = 0;
    if (vb + P < tiles) {
        tile_of(vb + P, tiles, tiles_m, tiles_n, group_m, tm_next, tn_next);
        tile_rows<C>(c, tm_next, tn_next, nGA, nGB, c.ksteps, c.kgroups, 0, lane, c.lo_next, c.hi_next, c.sc_next);
        c.knext = c.ksteps;
    }

    // every tile's first k-step starts its accumulators from 0 (FRESH, mfma_tile)
    v16f acc[C::kMB][C::kMA];
    v2u_t bias_bits[BIAS ? C::kMB * 4 : 1];
    if constexpr (BIAS) load_bias<C>(rBias, tn, wn, lane, bias_bits);

    // Prologue: steps 0-2 whole (a tile's first k-step does not issue step
    // 2's second part), all landed before the first k-step, so the first
    // tile's first two waits (which count past stores that this tile does not
    // have) wait for nothing.
    dma_part<C, 0, 0, 0, 0>(c, 0);
    dma_part<C, 0, 0, 1, 0>(c, 0);
    dma_part<C, 1, 1, 0, 0>(c, 1);
    dma_part<C, 1, 1, 1, 0>(c, 1);
    dma_part<C, 2, 2, 0, 0>(c, 2);
    dma_part<C, 2, 2, 1, 0>(c, 2);

    const Lds l = lds_offsets<C>(wave, lane);
    Regs<C> r;
    // vmcnt(0) as a builtin (not asm), so that the compiler's own wait
    // tracking also knows that nothing is outstanding past this point
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    __builtin_amdgcn_s_barrier();
    first_operands<C, 0>(r, l);

    for (;;) {
        // first period: its first two waits count past the previous tile's
        // stores and this tile's bias loads
        period<C, true, kFreshOps, false, 0>(c, 0, acc, r, l);
        // a period from k0 fetches steps k0+2 .. k0+kPeriod+2: all of this
        // tile while k0 + kPeriod + 2 < ksteps; the last one (or two) also
        // fetch the next tile's
        int k0 = C::kPeriod;
        if constexpr (C::Fmt::kInner)
            for (; k0 < c.kstream && k0 + C::kPeriod + 2 < c.ksteps; k0 += C::kPeriod)
                period<C, false, 0, true, 0>(c, k0, acc, r, l);
        for (; k0 < c.kstream; k0 += C::kPeriod) period<C, false, 0, false, 0>(c, k0, acc, r, l);
        // r now holds the next tile's first operands and scales
        if constexpr (BIAS) add_bias<C>(acc, bias_bits);
        store_tile_stream<C>(c, acc, tm, tn, M, N, rC, ldc, wave, lane);
        if constexpr (BIAS) {
            // The next tile's bias, after the stores in issue order as the
            // first waits assume.  (The compiler moves these loads past the
            // exit test below; its own wait before the first read of the
            // next tile then merges the paths with and without them and
            // comes out below the count, draining a few of the oldest
            // stores: correct, slightly conservative.)
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            load_bias<C>(rBias, tn_next, wn, lane, bias_bits);
            __builtin_amdgcn_sched_barrier(0);
        }
        vb += P;
        if (vb >= tiles) break;
        tm = tm_next;
        tn = tn_next;
#pragma unroll
        for (int q = 0; q < C::kLoLoads; ++q) c.lo_row[q] = c.lo_next[q];
        if constexpr (C::kHiLoads > 0) {
#pragma unroll
            for (int q = 0; q < C::kHiLoads; ++q) c.hi_off[q] = c.hi_next[q];
        }
#pragma unroll
        for (int q = 0; q < C::kScaleLoads; ++q) c.sc_row[q] = c.sc_next[q];
        c.knext = 0;
        if (vb + P < tiles) {
            tile_of(vb + P, tiles, tiles_m, tiles_n, group_m, tm_next, tn_next);
            tile_rows<C>(c, tm_next, tn_next, nGA, nGB, c.ksteps, c.kgroups, 0, lane, c.lo_next, c.hi_next,
                         c.sc_next);
            c.knext = c.ksteps;
        }
    }
    // drain the stores and the trailing (out-of-range) DMAs
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// ------------------------------------------------------------ FP8 (E5M2)
// The hybrid backward's GEMM: tensorwise E5M2 operands in the FP8 tiled
// layout (16-row groups, 64-element k-steps, 1 KB atoms; lane
// (r%16) + 16*((k%64)/16) owns 16 bytes), C = (A . B^T) * sa_inv * sb_inv.
// V_MFMA_SCALE_F32_32X32X64_F8F6F4 with both formats E5M2 and unit block
// scales (127): lane L of a 32-row operand tile supplies 32 bytes, row L%32,
// elements [32*(L/32), 32*(L/32) + 32) of the 64-wide step = two 16-byte
// slices of the atom, 256 bytes apart.  A 64-element step of a 16-row group
// is one 1 KB atom, as a 128-element MXFP4 step is, so the MXFP4
// configurations give the atom and DMA counts: the same workgroup shapes
// (256x256 main tiles; a last round that would fill at most half of the CUs
// as 128x128 tiles, as two K groups summed through LDS when those give at
// most one tile per CU), wave tiles, XCD order, LDS stages and epilogues
// (for bf16 output and short K, a persistent form with the wave-private
// epilogue of the block-scaled stream kernel); a stage holds one step, step
// k+3 is in flight while step k computes.
template <class S>
using Fp8Cfg = Cfg<Fp4Fmt, S>;
constexpr int kFmtBf8 = 1;          // MFMA f8f6f4 format code for E5M2
constexpr int kUnitScale = 127;     // E8M0 2^0
// Longest K of the persistent FP8 form: same box, bit-identical, the fc2
// dgrad (48 steps per tile) 0.548 -> 0.520 ms, the wgrad (288 steps, this K)
// a tie; longer K is not measured, so it keeps one tile per workgroup.
constexpr int64_t kFp8StreamKMax = 288 * 64;

template <int S, int G, class C>
__device__ __forceinline__ void fp8_dma_step(const Ctx<C, false> &c, int64_t k) {
#pragma unroll
    for (int r = 0; r < C::kLoLoads; ++r) {
        const int a = C::kWaves * r + c.wave;
        // plain-typed locals: a builtin call on template-dependent operands
        // does not resolve in the host compilation pass
        const __amdgpu_buffer_rsrc_t rsrc = a < C::kGA ? c.rA : c.rB;
        const uint32_t off =
            (k < c.ksteps ? (uint32_t)c.lo_row[r] + (uint32_t)(k * 1024) : kOutOfRange) + (uint32_t)c.lane16;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, MX_LDS((stage_buf<C, S, G>() + a * 1024)), 16, off, 0, 0, 0);
    }
}

// One k-step from stage S: wait until at most W of this wave's vector-memory
// instructions are outstanding (the step's own DMAs then have landed: by
// default the next two steps' DMAs may still be in flight), read the
// operands, issue the DMA of step kd of context cd into stage (S + 3) % 4,
// then the MFMAs.
template <class C, int S, int G, int W = 2 * C::kLoLoads>
__device__ __forceinline__ void fp8_step(const Ctx<C, false> &cd, int64_t kd, v16f (&acc)[C::kMB][C::kMA],
                                         int frag_off, int a_atom0, int b_atom0) {
    // this step's data landed for every wave, and every wave is done reading
    // the previous step's stage
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(W) : "memory");
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t *st = stage_buf<C, S, G>() + frag_off;
    uint4 bv[C::kMB][2], av[C::kMA][2];
#pragma unroll
    for (int i = 0; i < C::kMB; ++i) {
        bv[i][0] = *reinterpret_cast<const uint4 *>(st + (b_atom0 + 2 * i) * 1024);
        bv[i][1] = *reinterpret_cast<const uint4 *>(st + (b_atom0 + 2 * i) * 1024 + 256);
    }
#pragma unroll
    for (int j = 0; j < C::kMA; ++j) {
        av[j][0] = *reinterpret_cast<const uint4 *>(st + (a_atom0 + 2 * j) * 1024);
        av[j][1] = *reinterpret_cast<const uint4 *>(st + (a_atom0 + 2 * j) * 1024 + 256);
    }
    fp8_dma_step<(S + 3) & 3, G>(cd, kd);
#pragma unroll
    for (int i = 0; i < C::kMB; ++i) {
        const v8i bop = {(int)bv[i][0].x, (int)bv[i][0].y, (int)bv[i][0].z, (int)bv[i][0].w,
                         (int)bv[i][1].x, (int)bv[i][1].y, (int)bv[i][1].z, (int)bv[i][1].w};
#pragma unroll
        for (int j = 0; j < C::kMA; ++j) {
            const v8i aop = {(int)av[j][0].x, (int)av[j][0].y, (int)av[j][0].z, (int)av[j][0].w,
                             (int)av[j][1].x, (int)av[j][1].y, (int)av[j][1].z, (int)av[j][1].w};
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bop, aop, acc[i][j], kFmtBf8, kFmtBf8, 0,
                                                                        kUnitScale, 0, kUnitScale);
        }
    }
    // reads first (the MFMAs need them), each DMA after an MFMA
#pragma unroll
    for (int t = 0; t < C::kLoLoads; ++t) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
    if constexpr (C::kMA * C::kMB > C::kLoLoads)
        __builtin_amdgcn_sched_group_barrier(0x008, C::kMA * C::kMB - C::kLoLoads, 0);
}

// `steps` steps (a multiple of 4) of K group G's stages; steps past the
// group's own c.ksteps land as zeros.
template <class C, int G>
__device__ __forceinline__ void fp8_run(const Ctx<C, false> &c, v16f (&acc)[C::kMB][C::kMA], int64_t steps,
                                        int frag_off, int a_atom0, int b_atom0) {
    fp8_dma_step<0, G>(c, 0);
    fp8_dma_step<1, G>(c, 1);
    fp8_dma_step<2, G>(c, 2);
    for (int64_t k = 0; k < steps; k += 4) {
        fp8_step<C, 0, G>(c, k + 3, acc, frag_off, a_atom0, b_atom0);
        fp8_step<C, 1, G>(c, k + 4, acc, frag_off, a_atom0, b_atom0);
        fp8_step<C, 2, G>(c, k + 5, acc, frag_off, a_atom0, b_atom0);
        fp8_step<C, 3, G>(c, k + 6, acc, frag_off, a_atom0, b_atom0);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// One output tile per workgroup, 256x256 (workgroup b takes tile b of the
// XCD-remapped order) or 128x128 (workgroup b computes quarter b % 4 of
// 256x256 tile first + b / 4).  Split form: group g = wave / 4 takes steps
// [g * s0, ...) of K (s0 = half of them rounded up to a multiple of 4);
// both groups run s0 steps, so the per-step barriers line up, and group 1's
// partial tile is added into group 0's through LDS before the epilogue.
template <class C, bool OUT_BF16>
__global__ __launch_bounds__(C::kThreads) void gemm_fp8_kernel(int64_t M, int64_t N, int64_t K_pad, int tiles_m,
                                                               int tiles_n, int group_m, int first,
                                                               const uint8_t *__restrict__ A,
                                                               const float *__restrict__ a_scale_inv,
                                                               const uint8_t *__restrict__ B,
                                                               const float *__restrict__ b_scale_inv,
                                                               void *__restrict__ Cout, int64_t ldc) {
    constexpr bool kSplit = C::kKG == 2;
    const int lane = threadIdx.x & 63;
    const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // wave-uniform
    const int group = kSplit ? wave_all / C::kWaves : 0;
    const int wave = wave_all % C::kWaves;
    const int wm = wave % C::kWavesM, wn = wave / C::kWavesM;
    int tm, tn;
    if constexpr (C::kBM == 256) {
        tile_of(blockIdx.x, gridDim.x, tiles_m, tiles_n, group_m, tm, tn);
    } else {
        const int quarter = (int)(blockIdx.x & 3);
        tile_at(first + (int)(blockIdx.x >> 2), tiles_m, tiles_n, group_m, tm, tn);
        tm = 2 * tm + (quarter >> 1);
        tn = 2 * tn + (quarter & 1);
    }

    const int64_t ksteps = K_pad / 64;
    const int64_t s0 = kSplit ? 4 * cdiv(cdiv(ksteps, 2), 4) : ksteps;
    const int64_t kfirst = group ? s0 : 0;
    Ctx<C, false> c;
    c.ksteps = group ? ksteps - s0 : (s0 < ksteps ? s0 : ksteps);
    c.kgroups = 0;
    c.wave = wave;
    c.lane16 = lane * 16;
    c.lane4 = 0;
    const int64_t nGA = cdiv(M, 16), nGB = cdiv(N, 16);
    c.rA = make_rsrc(A, nGA * ksteps * 1024);
    c.rB = make_rsrc(B, nGB * ksteps * 1024);
    const int64_t gA0 = (int64_t)tm * C::kGA, gB0 = (int64_t)tn * C::kGB;
#pragma unroll
    for (int r = 0; r < C::kLoLoads; ++r) {
        const int a = C::kWaves * r + wave;
        const bool isA = a < C::kGA;
        int64_t g = isA ? gA0 + a : gB0 + (a - C::kGA);
        const int64_t gmax = (isA ? nGA : nGB) - 1;
        g = g < gmax ? g : gmax;
        c.lo_row[r] = (int)((g * ksteps + kfirst) * 1024);
    }
    const float scale = a_scale_inv[0] * b_scale_inv[0];

    v16f acc[C::kMB][C::kMA];
#pragma unroll
    for (int i = 0; i < C::kMB; ++i)
#pragma unroll
        for (int j = 0; j < C::kMA; ++j) acc[i][j] = v16f{};

    const int lrow = lane & 31, lhi = lane >> 5;
    const int frag_off = ((lrow >> 4) * 1024) + ((lrow & 15) + 32 * lhi) * 16;
    const int a_atom0 = wm * C::kTA, b_atom0 = C::kGA + wn * C::kTB;
    if (kSplit && group == 1) fp8_run<C, 1>(c, acc, s0, frag_off, a_atom0, b_atom0);
    else fp8_run<C, 0>(c, acc, s0, frag_off, a_atom0, b_atom0);

    if constexpr (kSplit) {
        // every wave is past its last stage read; group 1's stages take its partial tile
        __syncthreads();
        if (group == 1) {
#pragma unroll
            for (int i = 0; i < C::kMB; ++i)
#pragma unroll
                for (int j = 0; j < C::kMA; ++j) {
                    float *p = partial_slot<C>(wave, i * C::kMA + j) + lane;
#pragma unroll
                    for (int e = 0; e < 16; ++e) p[e * 64] = acc[i][j][e];
                }
        }
        __syncthreads();
        if (group == 0) {
#pragma unroll
            for (int i = 0; i < C::kMB; ++i)
#pragma unroll
                for (int j = 0; j < C::kMA; ++j) {
                    const float *p = partial_slot<C>(wave, i * C::kMA + j) + lane;
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][j][e] += p[e * 64];
                }
        }
    }
#pragma unroll
    for (int i = 0; i < C::kMB; ++i)
#pragma unroll
        for (int j = 0; j < C::kMA; ++j) acc[i][j] *= scale;
    store_tile<C, OUT_BF16>(acc, tm, tn, M, N, Cout, ldc, group, wave, wave_all, lane);
}

// Persistent form of the 256x256 FP8 kernel (bf16 output), as the
// block-scaled stream kernel: one workgroup per CU runs tiles b, b +
// gridDim.x, ... of the first `tiles` of the tile order as one stream of
// k-steps.  A tile is `steps` = ksteps rounded up to a multiple of 4 steps
// (at least 8), so every tile starts at stage 0; its last three steps issue
// the DMAs of the next tile's first three, and its epilogue stages C through
// stage 3 (the wave-private epilogue) while those land.  The stores are then
// in flight under the next tile's first steps: the first three waits count
// past the epi_stores() stores, the fourth needs them done.  Needs N % 8 == 0
// and M * ldc * 2 < 2^31 (32-bit store offsets).
template <class C>
__global__ __launch_bounds__(C::kThreads) void gemm_fp8_stream_kernel(int M, int N, int K_pad, int tiles_m,
                                                                      int tiles_n, int group_m, int tiles,
                                                                      const uint8_t *__restrict__ A,
                                                                      const float *__restrict__ a_scale_inv,
                                                                      const uint8_t *__restrict__ B,
                                                                      const float *__restrict__ b_scale_inv,
                                                                      void *__restrict__ Cout, int ldc) {
    static_assert(C::kKG == 1 && C::kBM == 256, "stream form: main tiles");
    constexpr int kWaitStores = 2 * C::kLoLoads + epi_stores<C>();
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % C::kWavesM, wn = wave / C::kWavesM;
    const int P = gridDim.x;
    const int ksteps = K_pad / 64;
    const int steps = 4 * ((ksteps + 3) / 4);
    const int nGA = (M + 15) / 16, nGB = (N + 15) / 16;
    Ctx<C, false> c;
    c.ksteps = ksteps;
    c.kgroups = 0;
    c.wave = wave;
    c.lane16 = lane * 16;
    c.lane4 = 0;
    c.rA = make_rsrc(A, (int64_t)nGA * ksteps * 1024);
    c.rB = make_rsrc(B, (int64_t)nGB * ksteps * 1024);
    Ctx<C, false> cn = c;   // the next tile's DMAs (ksteps 0: none left, out-of-range loads of zeros)
    const __amdgpu_buffer_rsrc_t rC = make_rsrc(Cout, (int64_t)M * ldc * 2);
    // byte offsets of this wave's unit rows (16-row groups, clamped to the last) at step 0
    const auto unit_rows = [&](int tm, int tn, int(&lo)[C::kLoLoads]) {
#pragma unroll
        for (int r = 0; r < C::kLoLoads; ++r) {
            const int a = C::kWaves * r + wave;
            const bool isA = a < C::kGA;
            const int g = isA ? tm * C::kGA + a : tn * C::kGB + (a - C::kGA);
            const int gmax = (isA ? nGA : nGB) - 1;
            lo[r] = (g < gmax ? g : gmax) * ksteps * 1024;
        }
    };
    int vb = blockIdx.x;
    int tm, tn, tm_next = 0, tn_next = 0;
    tile_of(vb, tiles, tiles_m, tiles_n, group_m, tm, tn);
    unit_rows(tm, tn, c.lo_row);
    cn.ksteps = 0;
    if (vb + P < tiles) {
        tile_of(vb + P, tiles, tiles_m, tiles_n, group_m, tm_next, tn_next);
        unit_rows(tm_next, tn_next, cn.lo_row);
        cn.ksteps = ksteps;
    }
    const float scale = a_scale_inv[0] * b_scale_inv[0];
    const int lrow = lane & 31, lhi = lane >> 5;
    const int frag_off = ((lrow >> 4) * 1024) + ((lrow & 15) + 32 * lhi) * 16;
    const int a_atom0 = wm * C::kTA, b_atom0 = C::kGA + wn * C::kTB;

    fp8_dma_step<0, 0>(c, 0);
    fp8_dma_step<1, 0>(c, 1);
    fp8_dma_step<2, 0>(c, 2);
    v16f acc[C::kMB][C::kMA];
    // one tile of the stream; FIRST: no stores of a previous tile are in flight
    const auto run = [&](auto first) {
#pragma unroll
        for (int i = 0; i < C::kMB; ++i)
#pragma unroll
            for (int j = 0; j < C::kMA; ++j) acc[i][j] = v16f{};
        // first period: steps 0-2 count past the previous tile's stores
        constexpr int kW0 = decltype(first)::value ? 2 * C::kLoLoads : kWaitStores;
        fp8_step<C, 0, 0, kW0>(c, 3, acc, frag_off, a_atom0, b_atom0);
        fp8_step<C, 1, 0, kW0>(c, 4, acc, frag_off, a_atom0, b_atom0);
        fp8_step<C, 2, 0, kW0>(c, 5, acc, frag_off, a_atom0, b_atom0);
        fp8_step<C, 3, 0>(c, 6, acc, frag_off, a_atom0, b_atom0);
        for (int k = 4; k < steps - 4; k += 4) {
            fp8_step<C, 0, 0>(c, k + 3, acc, frag_off, a_atom0, b_atom0);
            fp8_step<C, 1, 0>(c, k + 4, acc, frag_off, a_atom0, b_atom0);
            fp8_step<C, 2, 0>(c, k + 5, acc, frag_off, a_atom0, b_atom0);
            fp8_step<C, 3, 0>(c, k + 6, acc, frag_off, a_atom0, b_atom0);
        }
        // last period: its last three steps fetch the next tile's first three
        fp8_step<C, 0, 0>(c, steps - 1, acc, frag_off, a_atom0, b_atom0);
        fp8_step<C, 1, 0>(cn, 0, acc, frag_off, a_atom0, b_atom0);
        fp8_step<C, 2, 0>(cn, 1, acc, frag_off, a_atom0, b_atom0);
        fp8_step<C, 3, 0>(cn, 2, acc, frag_off, a_atom0, b_atom0);
#pragma unroll
        for (int i = 0; i < C::kMB; ++i)
#pragma unroll
            for (int j = 0; j < C::kMA; ++j) acc[i][j] *= scale;
        store_tile_private<C>(acc, tm, tn, M, N, rC, ldc, wave, lane);
    };
    // the first tile is peeled off the loop, so that every entry of the loop
    // has the previous tile's stores in flight
    run(std::true_type{});
    for (;;) {
        vb += P;
        if (vb >= tiles) break;
        tm = tm_next;
        tn = tn_next;
#pragma unroll
        for (int r = 0; r < C::kLoLoads; ++r) c.lo_row[r] = cn.lo_row[r];
        cn.ksteps = 0;
        if (vb + P < tiles) {
            tile_of(vb + P, tiles, tiles_m, tiles_n, group_m, tm_next, tn_next);
            unit_rows(tm_next, tn_next, cn.lo_row);
            cn.ksteps = ksteps;
        }
        run(std::false_type{});
    }
    // drain the stores and the trailing (out-of-range) DMAs
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// K == 0: C[i][j] = 0, or bias[j] (bf16 bits; exact in either output type).
template <typename T>
__global__ void fill_kernel(T *Cout, int64_t M, int64_t N, int64_t ldc, const uint16_t *bias) {
    const int64_t n = M * N;
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x) {
        const int64_t j = e % N;
        const uint16_t b = bias ? bias[j] : (uint16_t)0;
        if constexpr (sizeof(T) == 2) Cout[(e / N) * ldc + j] = b;
        else Cout[(e / N) * ldc + j] = __uint_as_float((uint32_t)b << 16);
    }
}

hipError_t launch_fill(int64_t M, int64_t N, const uint16_t *bias, mx_dtype out_dtype, void *Cout, int64_t ldc,
                       hipStream_t stream) {
    const int64_t blocks = cdiv(M * N, 256);
    const dim3 grid((unsigned)(blocks < 65536 ? (blocks > 0 ? blocks : 1) : 65536));
    if (out_dtype == MX_BF16)
        hipLaunchKernelGGL(fill_kernel<uint16_t>, grid, dim3(256), 0, stream, reinterpret_cast<uint16_t *>(Cout), M,
                           N, ldc, bias);
    else
        hipLaunchKernelGGL(fill_kernel<float>, grid, dim3(256), 0, stream, reinterpret_cast<float *>(Cout), M, N, ldc,
                           bias);
    return hipGetLastError();
}

// Tile rows per band of the tile order.  At any time an XCD's 32 CUs work on
// about 32 consecutive tiles of the order, which share A row blocks and B
// column blocks through its L2.  Same-box timings on MI355X: 4-row bands
// take 3-4% off the fc2 wgrad (12 x 48 tiles) and leave the 72-row shapes
// unchanged within 1%, where 8-row bands stay.
int band_rows(int tiles_m) { return tiles_m <= 16 ? 4 : 8; }

// The kernel instance for the output type and bias (HAS_BIAS false: the
// format's entry point takes no bias, so no bias instances exist).
template <class C, bool HAS_BIAS>
auto one_tile_kernel(bool bf, bool bias) {
    if constexpr (HAS_BIAS)
        return bf ? (bias ? gemm_kernel<C, true, true> : gemm_kernel<C, true, false>)
                  : (bias ? gemm_kernel<C, false, true> : gemm_kernel<C, false, false>);
    else
        return bf ? gemm_kernel<C, true, false> : gemm_kernel<C, false, false>;
}
template <class C, bool HAS_BIAS>
auto stream_kernel(bool bias) {
    if constexpr (HAS_BIAS) return bias ? gemm_stream_kernel<C, true> : gemm_stream_kernel<C, false>;
    else return gemm_stream_kernel<C, false>;
}

// Launch of one element format: main tiles (persistent form when it
// applies), then the leftover tiles of a last round that would fill at most
// 1 / tail_div of the CUs, as 128x128 tiles (the split form when they give
// at most one per CU and K has at least 8 k-steps).
template <class F, bool HAS_BIAS>
hipError_t launch_format(int64_t M, int64_t N, int64_t K_pad, int tail_div, const uint8_t *A, const uint8_t *As,
                         const uint8_t *B, const uint8_t *Bs, const uint16_t *bias, mx_dtype out_dtype, void *Cout,
                         int64_t ldc, hipStream_t stream) {
    using CM = Cfg<F, MainShape>;
    using CT = Cfg<F, TailShape>;
    using CS = Cfg<F, SplitShape>;
    const int tiles_m = (int)cdiv(M, 256), tiles_n = (int)cdiv(N, 256);
    const int tiles = tiles_m * tiles_n;
    const int group_m = band_rows(tiles_m);
    const int cus = device_cu_count();
    const int tail = (cus > 0 && tiles > cus && tiles % cus <= cus / tail_div) ? tiles % cus : 0;
    const bool bf = out_dtype == MX_BF16;
    const int64_t kgroups = cdiv(K_pad, 512);
    // Several tiles per workgroup: one persistent workgroup per CU.  Same-box
    // FP4 timings at 18432 rows: the stream form takes 7% off at 12-24
    // k-steps per tile and 3.5% at 48, ties at 96, and with its wave-private
    // epilogue takes 0.9% off at 144 (the fc2 wgrad).  Longer K is not
    // measured, so it keeps one tile per workgroup.
    bool streamed = false;
    if constexpr (F::kStream) {
        if (bf && N % 8 == 0 && M * ldc * 2 < (int64_t(1) << 31) && K_pad <= 144 * 128 && cus > 0 &&
            tiles - tail > cus && (4 * kgroups) % F::kPeriod == 0) {
            auto kernel = stream_kernel<CM, HAS_BIAS>(bias != nullptr);
            hipLaunchKernelGGL(kernel, dim3((unsigned)cus), dim3(CM::kThreads), 0, stream, (int)M, (int)N,
                               (int)K_pad, tiles_m, tiles_n, group_m, tiles - tail, A, As, B, Bs, bias, Cout,
                               (int)ldc);
            streamed = true;
        }
    }
    if (!streamed) {
        auto kernel = one_tile_kernel<CM, HAS_BIAS>(bf, bias != nullptr);
        hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles - tail)), dim3(CM::kThreads), 0, stream, M, N, K_pad,
                           tiles_m, tiles_n, group_m, 0, A, As, B, Bs, bias, Cout, ldc);
    }
    if (!tail) return hipGetLastError();
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int first = tiles - tail;
    // at most one 128x128 tile per CU (and K long enough to halve): the split form
    if (4 * tail <= cus && K_pad >= 8 * 128) {
        auto kernel = one_tile_kernel<CS, HAS_BIAS>(bf, bias != nullptr);
        hipLaunchKernelGGL(kernel, dim3((unsigned)(4 * tail)), dim3(CS::kThreads), 0, stream, M, N, K_pad, tiles_m,
                           tiles_n, group_m, first, A, As, B, Bs, bias, Cout, ldc);
    } else {
        auto kernel = one_tile_kernel<CT, HAS_BIAS>(bf, bias != nullptr);
        hipLaunchKernelGGL(kernel, dim3((unsigned)(4 * tail)), dim3(CT::kThreads), 0, stream, M, N, K_pad, tiles_m,
                           tiles_n, group_m, first, A, As, B, Bs, bias, Cout, ldc);
    }
    return hipGetLastError();
}

}  // namespace

// Compute units of the current device (cached per device; 0 if unknown).
int device_cu_count() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 0) n = 0;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

hipError_t launch_gemm(int64_t M, int64_t N, int64_t K, const uint8_t *A, const uint8_t *As,
                       const uint8_t *B, const uint8_t *Bs, const uint16_t *bias, mx_dtype out_dtype, void *C,
                       int64_t ldc, hipStream_t stream) {
    const int64_t K_pad = padded(K);
    if (K_pad == 0) return launch_fill(M, N, bias, out_dtype, C, ldc, stream);
    // buffer offsets are 32-bit: each operand blob (16-row groups of K_pad/2
    // bytes per row) must stay below 2 GiB
    if (cdiv(M, 16) * 16 * (K_pad / 2) >= (int64_t(1) << 31) || cdiv(N, 16) * 16 * (K_pad / 2) >= (int64_t(1) << 31))
        return hipErrorInvalidValue;
    // a last round that would fill at most half of the CUs goes to the tail
    // tiles (same-box A/B: larger thresholds lose)
    return launch_format<Fp4Fmt, true>(M, N, K_pad, 2, A, As, B, Bs, bias, out_dtype, C, ldc, stream);
}

hipError_t launch_gemm_fp6(int64_t M, int64_t N, int64_t K, int fmt_a, const uint8_t *A, const uint8_t *As,
                           int fmt_b, const uint8_t *B, const uint8_t *Bs, mx_dtype out_dtype, void *C, int64_t ldc,
                           hipStream_t stream) {
    const int64_t K_pad = padded(K);
    if (K_pad == 0) return launch_fill(M, N, nullptr, out_dtype, C, ldc, stream);
    // buffer offsets are 32-bit: each operand blob must stay below 2 GiB
    if (cdiv(M, 16) * (K_pad / 128) * 1536 >= (int64_t(1) << 31) ||
        cdiv(N, 16) * (K_pad / 128) * 1536 >= (int64_t(1) << 31))
        return hipErrorInvalidValue;
    // a last round that would fill at most a quarter of the CUs goes to the
    // tail tiles (same-box A/B on the fc2 shapes: 64 leftover tiles -7.5%; 96
    // no gain; 128 +1%)
    if (fmt_a == 2)
        return fmt_b == 2 ? launch_format<Fp6Fmt<2, 2>, false>(M, N, K_pad, 4, A, As, B, Bs, nullptr, out_dtype, C, ldc, stream)
                          : launch_format<Fp6Fmt<2, 3>, false>(M, N, K_pad, 4, A, As, B, Bs, nullptr, out_dtype, C, ldc, stream);
    return fmt_b == 2 ? launch_format<Fp6Fmt<3, 2>, false>(M, N, K_pad, 4, A, As, B, Bs, nullptr, out_dtype, C, ldc, stream)
                      : launch_format<Fp6Fmt<3, 3>, false>(M, N, K_pad, 4, A, As, B, Bs, nullptr, out_dtype, C, ldc, stream);
}

hipError_t launch_gemm_fp8(int64_t M, int64_t N, int64_t K, const uint8_t *A, const float *a_scale_inv,
                           const uint8_t *B, const float *b_scale_inv, mx_dtype out_dtype, void *C, int64_t ldc,
                           hipStream_t stream) {
    const int64_t K_pad = padded(K);
    if (K_pad == 0) return launch_fill(M, N, nullptr, out_dtype, C, ldc, stream);
    // buffer offsets are 32-bit: each operand blob must stay below 2 GiB
    if (cdiv(M, 16) * 16 * K_pad >= (int64_t(1) << 31) || cdiv(N, 16) * 16 * K_pad >= (int64_t(1) << 31))
        return hipErrorInvalidValue;
    using CM = Fp8Cfg<MainShape>;
    using CT = Fp8Cfg<TailShape>;
    using CS = Fp8Cfg<SplitShape>;
    const int tiles_m = (int)cdiv(M, 256), tiles_n = (int)cdiv(N, 256);
    const int tiles = tiles_m * tiles_n;
    const int group_m = band_rows(tiles_m);
    const int cus = device_cu_count();
    // a last round that would fill at most half of the CUs goes to the tail tiles
    const int tail = (cus > 0 && tiles > cus && tiles % cus <= cus / 2) ? tiles % cus : 0;
    const bool bf = out_dtype == MX_BF16;
    // several tiles per workgroup (persistent form): bf16 output, 8 to 288
    // steps per tile, more main tiles than CUs
    if (bf && N % 8 == 0 && M * ldc * 2 < (int64_t(1) << 31) && K_pad >= 8 * 64 && K_pad <= kFp8StreamKMax &&
        cus > 0 && tiles - tail > cus) {
        hipLaunchKernelGGL(gemm_fp8_stream_kernel<CM>, dim3((unsigned)cus), dim3(CM::kThreads), 0, stream, (int)M,
                           (int)N, (int)K_pad, tiles_m, tiles_n, group_m, tiles - tail, A, a_scale_inv, B, b_scale_inv,
                           C, (int)ldc);
    } else {
        auto main_kernel = bf ? gemm_fp8_kernel<CM, true> : gemm_fp8_kernel<CM, false>;
        hipLaunchKernelGGL(main_kernel, dim3((unsigned)(tiles - tail)), dim3(CM::kThreads), 0, stream, M, N, K_pad,
                           tiles_m, tiles_n, group_m, 0, A, a_scale_inv, B, b_scale_inv, C, ldc);
    }
    if (!tail) return hipGetLastError();
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int first = tiles - tail;
    // at most one 128x128 tile per CU and at least 16 steps: the split form
    if (4 * tail <= cus && K_pad >= 16 * 64) {
        auto kernel = bf ? gemm_fp8_kernel<CS, true> : gemm_fp8_kernel<CS, false>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(4 * tail)), dim3(CS::kThreads), 0, stream, M, N, K_pad, tiles_m,
                           tiles_n, group_m, first, A, a_scale_inv, B, b_scale_inv, C, ldc);
    } else {
        auto kernel = bf ? gemm_fp8_kernel<CT, true> : gemm_fp8_kernel<CT, false>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(4 * tail)), dim3(CT::kThreads), 0, stream, M, N, K_pad, tiles_m,
                           tiles_n, group_m, first, A, a_scale_inv, B, b_scale_inv, C, ldc);
    }
    return hipGetLastError();
}

}  // namespace mx
