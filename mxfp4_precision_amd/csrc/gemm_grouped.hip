// Block-scaled FP4 products grouped by expert, on the blobs of
// mx_quantize_grouped:
//   forward / dgrad: C[r][j] = sum_k A[r][k] B_e[j][k]  for the rows r of group e
//   wgrad:           C_e[i][j] = sum_r A[i][r] B[j][r]  over the rows r of group e
// The groups' ends are read on the device (grouped.h), so neither the grid
// nor the arguments depend on a routing result: the grid covers the most
// tiles that M rows in `groups` groups can need, and a workgroup past the
// tiles that there are returns.

#include "gemm_pipeline.h"
#include "grouped.h"
#include "grouped_forms.h"

namespace mx {
namespace {

// One output tile per workgroup.  Rows of C in no group are written as 0.
template <class C, bool OUT_BF16, bool BIAS>
__global__ __launch_bounds__(C::kThreads) void gemm_grouped_kernel(const int32_t *__restrict__ ends, int groups, int M,
                                                                   int N, int K_pad, int tiles_n,
                                                                   const uint8_t *__restrict__ A,
                                                                   const uint8_t *__restrict__ As,
                                                                   const uint8_t *__restrict__ B,
                                                                   const uint8_t *__restrict__ Bs,
                                                                   const uint16_t *__restrict__ bias,
                                                                   void *__restrict__ Cout, int64_t ldc) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int tm = 0, tn = 0;
    GroupPos p;
    const bool found = find_tile<C::kBM>(ends, groups, M, [&](int total_m) {
        const int id = xcd_position(blockIdx.x, total_m * tiles_n);
        if (id < 0) return -1;
        tile_at(id, total_m, tiles_n, total_m <= 16 ? 4 : 8, tm, tn);
        return tm;
    }, p);
    if (!found) return;

    v16f acc[C::kMB][C::kMA];
#pragma unroll
    for (int i = 0; i < C::kMB; ++i)
#pragma unroll
        for (int j = 0; j < C::kMA; ++j) acc[i][j] = v16f{};
    const bool live = p.group < groups;
    v2u_t bias_bits[BIAS ? C::kMB * 4 : 1];
    if constexpr (BIAS) {
        const uint16_t *b = bias + (int64_t)(live ? p.group : 0) * N;
        // (a group's bias starts at any even byte, so it is read by element)
        const int col0 = tn * C::kBN + (wave / C::kWavesM) * C::kWN + 4 * (lane >> 5);
#pragma unroll
        for (int i = 0; i < C::kMB; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t v[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int col = col0 + 32 * i + 8 * q + t;
                    v[t] = live && col < N ? b[col] : 0;
                }
                bias_bits[i * 4 + q] = v2u_t{v[0] | (v[1] << 16), v[2] | (v[3] << 16)};
            }
    }
    const int64_t ksteps = K_pad / 128, kgroups = cdiv(K_pad, 512);
    if (live && ksteps > 0) {
        Ctx<C, false> c;
        c.ksteps = ksteps;
        c.kgroups = kgroups;
        c.wave = wave;
        c.lane16 = lane * 16;
        c.lane4 = lane * 4;
        const int64_t nGA = cdiv(p.rows, 16), nGB = cdiv(N, 16);
        c.rA = make_rsrc(A + (int64_t)p.r16 * ksteps * 1024, nGA * ksteps * 1024);
        c.rB = make_rsrc(B + p.group * (nGB * ksteps * 1024), nGB * ksteps * 1024);
        c.rAs = make_rsrc(As + (int64_t)p.r16 * kgroups * 256, nGA * kgroups * 256);
        c.rBs = make_rsrc(Bs + p.group * (nGB * kgroups * 256), nGB * kgroups * 256);
        tile_rows<C>(c, p.tile, tn, nGA, nGB, ksteps, kgroups, 0, lane, c.lo_row, c.hi_off, c.sc_row);
        const Lds l = lds_offsets<C>(wave, lane);
        run_tile<C, 0>(c, acc, l, 4 * kgroups);
    }
    if constexpr (BIAS) add_bias<C>(acc, bias_bits);
    store_tile<C, OUT_BF16>(acc, p.tile, tn, p.rows, N,
                            reinterpret_cast<uint8_t *>(Cout) + (int64_t)p.start * ldc * (OUT_BF16 ? 2 : 4), ldc, 0,
                            wave, wave, lane);
}

// ------------------------------------------------------------ few rows
// Groups of few rows (decoding): what counts is reading the weights once and
// the latency of one pass, so B does not go through LDS.  An atom (16 rows x
// 128 k) is exactly the operand of V_MFMA_SCALE_F32_16X16X128_F8F6F4: lane L
// holds row L % 16, block L / 16, 16 bytes at 16 L, and loads them straight
// into registers.  A workgroup's tile is 64 rows (or the group's remainder,
// MA atoms) x 32 columns; its four waves take k-step 4 h + wave of every
// k-group h, so each reads one byte of the scale dwords that all four load,
// and their sums are added in wave order through LDS.  Up to eight k-groups
// are in flight per wave.  192 rows in 32 groups, N 1536, K 4096: 17 us, 6.2 TB/s
// of weights (128x128 tiles 19); two or four k-groups in flight, 16 or 64
// columns and non-temporal loads are no faster.
template <int MA, int DEPTH>
__device__ __forceinline__ void few_rows_sum(__amdgpu_buffer_rsrc_t rA, __amdgpu_buffer_rsrc_t rAs,
                                             __amdgpu_buffer_rsrc_t rB, __amdgpu_buffer_rsrc_t rBs, int gA0, int nGA,
                                             int gB0, int nGB, int ksteps, int kgroups, int wave, int lane,
                                             v4f (&acc)[kFewM / 16][kFewNB], int h0 = 0) {
    // atom rows past an operand are clamped to its last one: those results are not stored
    int a_row[MA], b_row[kFewNB];
#pragma unroll
    for (int i = 0; i < MA; ++i) a_row[i] = min(gA0 + i, nGA - 1);
#pragma unroll
    for (int j = 0; j < kFewNB; ++j) b_row[j] = min(gB0 + j, nGB - 1);
    const uint32_t lane16 = (uint32_t)lane * 16, lane4 = (uint32_t)lane * 4;
    for (; h0 + DEPTH <= kgroups; h0 += DEPTH) {
        v4u_t a[DEPTH][MA], b[DEPTH][kFewNB];
        uint32_t as[DEPTH][MA], bs[DEPTH][kFewNB];
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            const int h = h0 + u, ks = 4 * h + wave;
            // Past K the data read as zeros: the lane offset is out of range on
            // its own, the scalar one is then 0 (the range check subtracts it
            // from the range).
            const bool in = ks < ksteps;
            const uint32_t off = in ? lane16 : kOutOfRange;
#pragma unroll
            for (int j = 0; j < kFewNB; ++j) {
                b[u][j] = __builtin_amdgcn_raw_buffer_load_b128(rB, off, in ? (b_row[j] * ksteps + ks) * 1024 : 0, 0);
                bs[u][j] = __builtin_amdgcn_raw_buffer_load_b32(rBs, lane4, (b_row[j] * kgroups + h) * 256, 0);
            }
#pragma unroll
            for (int i = 0; i < MA; ++i) {
                a[u][i] = __builtin_amdgcn_raw_buffer_load_b128(rA, off, in ? (a_row[i] * ksteps + ks) * 1024 : 0, 0);
                as[u][i] = __builtin_amdgcn_raw_buffer_load_b32(rAs, lane4, (a_row[i] * kgroups + h) * 256, 0);
            }
        }
#pragma unroll
        for (int u = 0; u < DEPTH; ++u)
#pragma unroll
            for (int i = 0; i < MA; ++i)
#pragma unroll
                for (int j = 0; j < kFewNB; ++j) {
                    const v8i bop = {(int)b[u][j][0], (int)b[u][j][1], (int)b[u][j][2], (int)b[u][j][3], 0, 0, 0, 0};
                    const v8i aop = {(int)a[u][i][0], (int)a[u][i][1], (int)a[u][i][2], (int)a[u][i][3], 0, 0, 0, 0};
                    const int sb = (int)(bs[u][j] >> (8 * wave)), sa = (int)(as[u][i] >> (8 * wave));
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bop, aop, acc[i][j], Fp4Fmt::kFb,
                                                                                 Fp4Fmt::kFa, 0, sb, 0, sa);
                }
    }
    // the k-groups left over, half as many at a time
    if constexpr (DEPTH > 1)
        few_rows_sum<MA, DEPTH / 2>(rA, rAs, rB, rBs, gA0, nGA, gB0, nGB, ksteps, kgroups, wave, lane, acc, h0);
}

template <bool OUT_BF16, bool BIAS>
__global__ __launch_bounds__(256) void gemm_grouped_few_kernel(const int32_t *__restrict__ ends, int groups, int M,
                                                               int N, int K_pad, int tiles_n,
                                                               const uint8_t *__restrict__ A,
                                                               const uint8_t *__restrict__ As,
                                                               const uint8_t *__restrict__ B,
                                                               const uint8_t *__restrict__ Bs,
                                                               const uint16_t *__restrict__ bias,
                                                               void *__restrict__ Cout, int64_t ldc) {
    constexpr int kTiles = kFewM / 16 * kFewNB;
    __shared__ v4f s_sum[4][kTiles][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int tn = 0;
    GroupPos p;
    const bool found = find_tile<kFewM>(ends, groups, M, [&](int total_m) {
        const int id = xcd_position(blockIdx.x, total_m * tiles_n);
        if (id < 0) return -1;
        tn = id % tiles_n;
        return id / tiles_n;
    }, p);
    if (!found) return;
    const bool live = p.group < groups;
    const int row0 = p.tile * kFewM;
    const int ma = min((p.rows - row0 + 15) / 16, kFewM / 16);
    v4f acc[kFewM / 16][kFewNB];
#pragma unroll
    for (int i = 0; i < kFewM / 16; ++i)
#pragma unroll
        for (int j = 0; j < kFewNB; ++j) acc[i][j] = v4f{};
    const int ksteps = K_pad / 128, kgroups = (K_pad + 511) / 512;
    if (live && ksteps > 0) {
        const int nGA = (p.rows + 15) / 16, nGB = (N + 15) / 16;
        const int64_t gB = (int64_t)p.group * nGB;
        const auto rA = make_rsrc(A + (int64_t)p.r16 * ksteps * 1024, (int64_t)nGA * ksteps * 1024);
        const auto rAs = make_rsrc(As + (int64_t)p.r16 * kgroups * 256, (int64_t)nGA * kgroups * 256);
        const auto rB = make_rsrc(B + gB * ksteps * 1024, (int64_t)nGB * ksteps * 1024);
        const auto rBs = make_rsrc(Bs + gB * kgroups * 256, (int64_t)nGB * kgroups * 256);
        const int gA0 = row0 / 16, gB0 = tn * kFewNB;
        if (ma == 1) few_rows_sum<1, 8>(rA, rAs, rB, rBs, gA0, nGA, gB0, nGB, ksteps, kgroups, wave, lane, acc);
        else if (ma == 2) few_rows_sum<2, 4>(rA, rAs, rB, rBs, gA0, nGA, gB0, nGB, ksteps, kgroups, wave, lane, acc);
        else few_rows_sum<4, 4>(rA, rAs, rB, rBs, gA0, nGA, gB0, nGB, ksteps, kgroups, wave, lane, acc);
    }
#pragma unroll
    for (int i = 0; i < kFewM / 16; ++i)
#pragma unroll
        for (int j = 0; j < kFewNB; ++j)
            if (i < ma) s_sum[wave][i * kFewNB + j][lane] = acc[i][j];
    __syncthreads();
    // lane L of tile (i, j): row 16 i + L % 16, columns 16 j + 4 (L / 16) + 0..3
    for (int t = wave; t < ma * kFewNB; t += 4) {
        v4f v = s_sum[0][t][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            const v4f q = s_sum[w][t][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += q[e];
        }
        const int row = row0 + 16 * (t / kFewNB) + (lane & 15);
        const int col = tn * kFewN + 16 * (t % kFewNB) + 4 * (lane >> 4);
        if (row >= p.rows || col >= N) continue;
        if constexpr (BIAS) {
            if (live) {
                const uint16_t *b = bias + (int64_t)p.group * N + col;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (col + e < N) v[e] += __uint_as_float((uint32_t)b[e] << 16);
            }
        }
        const int64_t at = ((int64_t)p.start + row) * ldc + col;
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

// wgrad: workgroup -> (group, tile of its M x N product); K = the group's rows.
template <class C, bool OUT_BF16>
__global__ __launch_bounds__(C::kThreads) void gemm_grouped_wgrad_kernel(const int32_t *__restrict__ ends, int groups,
                                                                         int rows, int M, int N, int tiles_m,
                                                                         int tiles_n, const uint8_t *__restrict__ A,
                                                                         const uint8_t *__restrict__ As,
                                                                         const uint8_t *__restrict__ B,
                                                                         const uint8_t *__restrict__ Bs,
                                                                         void *__restrict__ Cout, int64_t ldc,
                                                                         int64_t group_stride) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per_group = tiles_m * tiles_n;
    const int id = xcd_position(blockIdx.x, groups * per_group);
    if (id < 0) return;
    const int e = id / per_group;
    const GroupPos p = find_group(ends, groups, rows, e);
    int tm, tn;
    tile_at(id - e * per_group, tiles_m, tiles_n, tiles_m <= 16 ? 4 : 8, tm, tn);

    v16f acc[C::kMB][C::kMA];
#pragma unroll
    for (int i = 0; i < C::kMB; ++i)
#pragma unroll
        for (int j = 0; j < C::kMA; ++j) acc[i][j] = v16f{};
    if (p.rows > 0) {
        Ctx<C, false> c;
        c.ksteps = units(p.rows, 128);
        c.kgroups = units(p.rows, 512);
        c.wave = wave;
        c.lane16 = lane * 16;
        c.lane4 = lane * 4;
        const int64_t nGA = cdiv(M, 16), nGB = cdiv(N, 16);
        c.rA = make_rsrc(A + p.k128 * (nGA * 1024), nGA * c.ksteps * 1024);
        c.rB = make_rsrc(B + p.k128 * (nGB * 1024), nGB * c.ksteps * 1024);
        c.rAs = make_rsrc(As + p.k512 * (nGA * 256), nGA * c.kgroups * 256);
        c.rBs = make_rsrc(Bs + p.k512 * (nGB * 256), nGB * c.kgroups * 256);
        tile_rows<C>(c, tm, tn, nGA, nGB, c.ksteps, c.kgroups, 0, lane, c.lo_row, c.hi_off, c.sc_row);
        const Lds l = lds_offsets<C>(wave, lane);
        run_tile<C, 0>(c, acc, l, 4 * c.kgroups);
    }
    store_tile<C, OUT_BF16>(acc, tm, tn, M, N,
                            reinterpret_cast<uint8_t *>(Cout) + e * group_stride * (OUT_BF16 ? 2 : 4), ldc, 0, wave,
                            wave, lane);
}

// ------------------------------------------------------------ persistent form
// One workgroup per CU runs its 256x256 tiles as one stream of k-steps, as
// the persistent form of gemm.hip does (the next tile's first steps are
// fetched during the current tile's last ones, the stores drain while the
// next tile computes).  Here the next tile may lie in another group: every
// offset counts from the whole blob (both blobs below 2 GiB), so crossing a
// group changes scalars only, and with WGRAD a tile's number of k-steps
// changes too.  What a tile needs of its group is looked up in a table that
// the workgroup builds in LDS at its start: at 16-32 k-steps per tile the
// ends' load and scan in front of each tile cost about a tenth of it.  A tile
// without k-steps (rows in no group; a group without rows) runs one k-group
// of zeros.
//
// An XCD's workgroups walk a contiguous range of the tile order round-robin,
// so that they share A rows and B columns in its L2.  The ranges hold equally
// many tiles, or, with WGRAD, equally much work: a tile costs its k-steps and
// kTileCost more for its stores.  Training steps of 16384 rows in 16 groups
// (416 us) and 65536 in 32 (1235), run in turn with others: kTileCost 8 takes 2.4
// and 0.5% more, 0 takes 0.7% less and 0.9% more, equally many tiles 5% more.
constexpr int kTileCost = 4;

struct StreamTile {
    int ksteps;      // 0: zeros
    int tn, rows;    // column tile; rows of C that the tile has
    int64_t base;    // element of C where the tile's first row starts
    int bias;        // index of its group's bias, or -1
};

// v, as a value that the compiler does not compute ahead of a loop and hold:
// the k-loop leaves no registers for that.
__device__ __forceinline__ int hidden(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

template <class C, bool WGRAD, bool BIAS, bool ODD>
__global__ __launch_bounds__(C::kThreads) void gemm_grouped_stream_kernel(
    const int32_t *__restrict__ ends, int groups, int grows, int M, int N, int K_pad, int tiles_m, int tiles_n,
    const uint8_t *__restrict__ A, const uint8_t *__restrict__ As, const uint8_t *__restrict__ B,
    const uint8_t *__restrict__ Bs, const uint16_t *__restrict__ bias, uint16_t *__restrict__ Cout, int ldc,
    int64_t group_stride) {
    // groups: {tiles, or work, of the groups so far; first row; rows; blob units before it}
    __shared__ int4 s_group[kStreamGroups + 1];
    __shared__ int s_k512[WGRAD ? kStreamGroups : 1];
    constexpr int kBiasLoads = BIAS ? C::kMB * 4 : 0;
    constexpr int kFreshOps = epi_stores<C>() + kBiasLoads;
    constexpr int kBlob = 0x7FFFFFFF;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave / C::kWavesM;

    if (wave == 0) {
        GroupCarry c;
        int work = 0;
        for (int base = 0; base < groups; base += 64) {
            const GroupLane g = group_block<C::kBM, true>(ends, groups, grows, base, lane, c);
            int sum = g.tiles, before = g.r16 - units(g.rows, 16);
            if constexpr (WGRAD) {
                const int kg = units(g.rows, 512);
                sum = work + wave_scan<false>(base + lane < groups ? 4 * max(kg, 1) + kTileCost : 0);
                work = __builtin_amdgcn_readlane(sum, 63);
                before = g.k128 - units(g.rows, 128);
                if (base + lane < groups) s_k512[base + lane] = g.k512 - kg;
            }
            if (base + lane < groups) s_group[base + lane] = int4{sum, g.start, g.rows, before};
        }
        const int rest = grows - c.end;
        if (!WGRAD && lane == 0) s_group[groups] = int4{c.tiles + units(rest, C::kBM), c.end, rest, 0};
    }
    __syncthreads();

    // the group whose running sum passes v, and its entry
    const auto find = [&](int v, int last, int &e, int4 &g) {
        int lane = hidden(threadIdx.x & 63);
        for (int base = 0;; base += 64) {
            const int4 mine = s_group[min(base + lane, last)];
            const uint64_t past = __builtin_amdgcn_ballot_w64(v < mine.x || base + lane >= last);
            if (past) {
                const int l = __builtin_ctzll(past);
                e = base + l;
                g = int4{__builtin_amdgcn_readlane(mine.x, l), __builtin_amdgcn_readlane(mine.y, l),
                         __builtin_amdgcn_readlane(mine.z, l), __builtin_amdgcn_readlane(mine.w, l)};
                return;
            }
        }
    };
    int total, at, stop;   // tiles; this workgroup's next one and its XCD's end
    const int xcd = blockIdx.x % kXcds, step = gridDim.x / kXcds;
    if constexpr (WGRAD) {
        tiles_m = (M + C::kBM - 1) / C::kBM;
        const int per = tiles_m * tiles_n;
        total = groups * per;
        const int64_t work = __builtin_amdgcn_readfirstlane(s_group[groups - 1].x);
        const auto first_of = [&](int x) {
            if (x == 0) return 0;
            if (x == kXcds) return total;
            const int v = (int)(work * x / kXcds);
            int e;
            int4 g;
            find(v, groups - 1, e, g);
            const int cost = 4 * max(units(g.z, 512), 1) + kTileCost;
            return e * per + (int)((int64_t)(v - (g.x - cost)) * per / cost);
        };
        at = first_of(xcd);
        stop = first_of(xcd + 1);
    } else {
        tiles_m = __builtin_amdgcn_readfirstlane(s_group[groups].x);
        total = tiles_m * tiles_n;
        at = (int)((int64_t)total * xcd / kXcds);
        stop = (int)((int64_t)total * (xcd + 1) / kXcds);
    }
    at = __builtin_amdgcn_readfirstlane(at + (int)(blockIdx.x / kXcds));
    stop = __builtin_amdgcn_readfirstlane(stop);
    if (at >= stop) return;

    Ctx<C, true> c;
    c.wave = wave;
    c.lane16 = lane * 16;
    c.lane4 = lane * 4;
    c.rA = make_rsrc(A, kBlob);
    c.rB = make_rsrc(B, kBlob);
    c.rAs = make_rsrc(As, kBlob);
    c.rBs = make_rsrc(Bs, kBlob);
    const int nGB = (N + 15) / 16;
    // tile `id`: its values, and the blob offsets of this wave's DMA units
    const auto resolve = [&](int id, StreamTile &t, int (&lo)[C::kLoLoads], int (&sc)[C::kScaleLoads]) {
        int tm, nGA, lo_a, lo_b, sc_a, sc_b, kgroups, e;   // blob offsets of the group
        int4 g;
        if constexpr (WGRAD) {
            const int per = tiles_m * tiles_n;
            e = id / per;
            const int4 v = s_group[e];
            g = int4{0, 0, __builtin_amdgcn_readfirstlane(v.z), __builtin_amdgcn_readfirstlane(v.w)};
            const int k512 = __builtin_amdgcn_readfirstlane(s_k512[e]);
            tile_at(id - e * per, tiles_m, tiles_n, tiles_m <= 16 ? 4 : 8, tm, t.tn);
            t.ksteps = units(g.z, 128);
            kgroups = units(g.z, 512);
            nGA = (M + 15) / 16;
            lo_a = g.w * nGA * 1024;
            lo_b = g.w * nGB * 1024;
            sc_a = k512 * nGA * 256;
            sc_b = k512 * nGB * 256;
            t.rows = M - tm * C::kBM;
            t.base = e * group_stride + (int64_t)tm * C::kBM * ldc;
        } else {
            tile_at(id, tiles_m, tiles_n, tiles_m <= 16 ? 4 : 8, tm, t.tn);
            find(tm, groups, e, g);
            tm -= g.x - units(g.z, C::kBM);
            t.ksteps = e < groups ? K_pad / 128 : 0;
            kgroups = units(K_pad, 512);
            nGA = units(g.z, 16);
            lo_a = g.w * t.ksteps * 1024;
            sc_a = g.w * kgroups * 256;
            lo_b = e * nGB * t.ksteps * 1024;
            sc_b = e * nGB * kgroups * 256;
            t.rows = g.z - tm * C::kBM;
            t.base = (int64_t)(g.y + tm * C::kBM) * ldc;
        }
        t.bias = e < groups ? e : -1;
        // (all of it is uniform, which the compiler does not see through the
        // table: in vector registers it would spill the k-loop)
        const auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
        t.ksteps = uniform(t.ksteps);
        t.tn = uniform(t.tn);
        t.rows = uniform(t.rows);
        t.bias = uniform(t.bias);
        t.base = (int64_t)(((uint64_t)(uint32_t)uniform((int)(t.base >> 32)) << 32) | (uint32_t)uniform((int)t.base));
        // row groups past an operand are clamped to its last one: those rows of C are not stored
#pragma unroll
        for (int r = 0; r < C::kLoLoads; ++r) {
            const bool isA = C::kWaves * (r + 1) <= C::kGA;
            const int a = C::kWaves * r + wave;
            const int row = isA ? min(tm * C::kGA + a, nGA - 1) : min(t.tn * C::kGB + a - C::kGA, nGB - 1);
            lo[r] = uniform((isA ? lo_a : lo_b) + row * t.ksteps * 1024);
            sc[r] = uniform((isA ? sc_a : sc_b) + row * kgroups * 256);
        }
    };
    static_assert(C::kLoLoads == C::kScaleLoads && C::kHiLoads == 0, "one offset each per unit");
    const auto bias_of = [&](const StreamTile &t) {
        return make_rsrc(bias + (int64_t)(t.bias > 0 ? t.bias : 0) * N, t.bias < 0 ? 0 : (N * 2 + 15) / 16 * 16);
    };
    const auto start_tile = [&](const StreamTile &t) {
        c.ksteps = t.ksteps;
        c.kgroups = (t.ksteps + 3) / 4;
        c.kstream = 4 * max(c.kgroups, 1);
    };

    StreamTile cur, next{};
    resolve(at, cur, c.lo_row, c.sc_row);
    start_tile(cur);
    c.knext = 0;
    at += step;
    if (at < stop) {
        resolve(at, next, c.lo_next, c.sc_next);
        c.knext = next.ksteps;
    }
    v16f acc[C::kMB][C::kMA];
    v2u_t bias_bits[BIAS ? C::kMB * 4 : 1];
    if constexpr (BIAS) load_bias<C>(bias_of(cur), cur.tn, wn, lane, bias_bits);

    // as in the ungrouped persistent form: steps 0-2 whole, all landed before the first k-step
    dma_part<C, 0, 0, 0, 0>(c, 0);
    dma_part<C, 0, 0, 1, 0>(c, 0);
    dma_part<C, 1, 1, 0, 0>(c, 1);
    dma_part<C, 1, 1, 1, 0>(c, 1);
    dma_part<C, 2, 2, 0, 0>(c, 2);
    dma_part<C, 2, 2, 1, 0>(c, 2);
    const Lds l = lds_offsets<C>(wave, lane);
    Regs<C> r;
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    __builtin_amdgcn_s_barrier();
    first_operands<C, 0>(r, l);

    for (;;) {
        period<C, true, kFreshOps, false, 0>(c, 0, acc, r, l);
        int k0 = C::kPeriod;
        for (; k0 + C::kPeriod + 2 < c.ksteps; k0 += C::kPeriod) period<C, false, 0, true, 0>(c, k0, acc, r, l);
        for (; k0 < c.kstream; k0 += C::kPeriod) period<C, false, 0, false, 0>(c, k0, acc, r, l);
        if constexpr (BIAS) add_bias<C>(acc, bias_bits);
        dma_part<C, 2, 2, 1, 0>(c, c.kstream + 2);
        store_tile_private<C, ODD>(acc, 0, cur.tn, cur.rows, N, make_rsrc(Cout + cur.base, kBlob), ldc, wave,
                                   hidden(lane));
        if constexpr (BIAS) {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            load_bias<C>(bias_of(next), next.tn, wn, lane, bias_bits);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (at >= stop) break;
        at += step;
        cur = next;
        start_tile(cur);
#pragma unroll
        for (int q = 0; q < C::kLoLoads; ++q) c.lo_row[q] = c.lo_next[q];
#pragma unroll
        for (int q = 0; q < C::kScaleLoads; ++q) c.sc_row[q] = c.sc_next[q];
        c.knext = 0;
        if (at < stop) {
            resolve(at, next, c.lo_next, c.sc_next);
            c.knext = next.ksteps;
        }
    }
    // drain the stores and the trailing (out-of-range) DMAs
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <class S>
hipError_t launch_shape(const GroupedGemmArgs &a, hipStream_t stream) {
    using C = Cfg<Fp4Fmt, S>;
    const int tiles_n = (int)cdiv(a.N, C::kBN);
    const int64_t blocks = cdiv(max_tiles(a.M, a.groups, C::kBM) * tiles_n, kXcds) * kXcds;
    const bool bf = a.out_dtype == MX_BF16;
    auto kernel = bf ? (a.bias ? gemm_grouped_kernel<C, true, true> : gemm_grouped_kernel<C, true, false>)
                     : (a.bias ? gemm_grouped_kernel<C, false, true> : gemm_grouped_kernel<C, false, false>);
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(C::kThreads), 0, stream, a.ends, a.groups, (int)a.M,
                       (int)a.N, (int)padded(a.K), tiles_n, a.A, a.As, a.B, a.Bs, a.bias, a.C, a.ldc);
    return hipGetLastError();
}

hipError_t launch_few(const GroupedGemmArgs &a, hipStream_t stream) {
    const int tiles_n = (int)cdiv(a.N, kFewN);
    const int64_t blocks = cdiv(max_tiles(a.M, a.groups, kFewM) * tiles_n, kXcds) * kXcds;
    const bool bf = a.out_dtype == MX_BF16;
    auto kernel = bf ? (a.bias ? gemm_grouped_few_kernel<true, true> : gemm_grouped_few_kernel<true, false>)
                     : (a.bias ? gemm_grouped_few_kernel<false, true> : gemm_grouped_few_kernel<false, false>);
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a.ends, a.groups, (int)a.M, (int)a.N,
                       (int)padded(a.K), tiles_n, a.A, a.As, a.B, a.Bs, a.bias, a.C, a.ldc);
    return hipGetLastError();
}

hipError_t launch_stream(const GroupedGemmArgs &a, int cus, hipStream_t stream) {
    using C = Cfg<Fp4Fmt, MainShape>;
    auto kernel = odd_rows(a, a.N) ? (a.bias ? gemm_grouped_stream_kernel<C, false, true, true>
                                             : gemm_grouped_stream_kernel<C, false, false, true>)
                                   : (a.bias ? gemm_grouped_stream_kernel<C, false, true, false>
                                             : gemm_grouped_stream_kernel<C, false, false, false>);
    hipLaunchKernelGGL(kernel, dim3((unsigned)cus), dim3(C::kThreads), 0, stream, a.ends, a.groups, (int)a.M, (int)a.M,
                       (int)a.N, (int)padded(a.K), 0, (int)cdiv(a.N, C::kBN), a.A, a.As, a.B, a.Bs, a.bias,
                       static_cast<uint16_t *>(a.C), (int)a.ldc, int64_t(0));
    return hipGetLastError();
}

hipError_t launch_wgrad_stream(const GroupedGemmArgs &a, int cus, hipStream_t stream) {
    using C = Cfg<Fp4Fmt, MainShape>;
    auto kernel = wgrad_odd_rows(a) ? gemm_grouped_stream_kernel<C, true, false, true>
                                                               : gemm_grouped_stream_kernel<C, true, false, false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)cus), dim3(C::kThreads), 0, stream, a.ends, a.groups, (int)a.M, (int)a.N,
                       (int)a.K, 0, 0, (int)cdiv(a.K, C::kBN), a.A, a.As, a.B, a.Bs, a.bias,
                       static_cast<uint16_t *>(a.C), (int)a.ldc, a.group_stride);
    return hipGetLastError();
}

template <class S>
hipError_t launch_wgrad_shape(const GroupedGemmArgs &a, hipStream_t stream) {
    using C = Cfg<Fp4Fmt, S>;
    const int tiles_m = (int)cdiv(a.N, C::kBM), tiles_n = (int)cdiv(a.K, C::kBN);
    const int64_t blocks = cdiv((int64_t)a.groups * tiles_m * tiles_n, kXcds) * kXcds;
    auto kernel = a.out_dtype == MX_BF16 ? gemm_grouped_wgrad_kernel<C, true> : gemm_grouped_wgrad_kernel<C, false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(C::kThreads), 0, stream, a.ends, a.groups, (int)a.M,
                       (int)a.N, (int)a.K, tiles_m, tiles_n, a.A, a.As, a.B, a.Bs, a.C, a.ldc, a.group_stride);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_grouped(const GroupedGemmArgs &a, hipStream_t stream) {
    const int cus = device_cu_count() / kXcds * kXcds;
    switch (gemm_form(a, cus)) {
    case GemmForm::kFewRows: return launch_few(a, stream);
    case GemmForm::kTiles128: return launch_shape<TailShape>(a, stream);
    case GemmForm::kPersistent: return launch_stream(a, cus, stream);
    case GemmForm::kTiles256: break;
    }
    return launch_shape<MainShape>(a, stream);
}

hipError_t launch_gemm_grouped_wgrad(const GroupedGemmArgs &a, hipStream_t stream) {
    const int cus = device_cu_count() / kXcds * kXcds;
    switch (wgrad_form(a, cus)) {
    case GemmForm::kTiles128: return launch_wgrad_shape<TailShape>(a, stream);
    case GemmForm::kPersistent: return launch_wgrad_stream(a, cus, stream);
    default: return launch_wgrad_shape<MainShape>(a, stream);
    }
}

}  // namespace mx
