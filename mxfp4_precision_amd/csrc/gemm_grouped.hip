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

namespace mx {
namespace {

typedef int v4i_t __attribute__((ext_vector_type(4)));

// Tile `b` of `total` in XCD-contiguous order, or -1 (a workgroup past its
// XCD's share).
__device__ __forceinline__ int xcd_position(int b, int total) {
    const int xcd = b % kXcds, local = b / kXcds;
    const int per = total / kXcds, rem = total % kXcds;
    if (local >= per + (xcd < rem ? 1 : 0)) return -1;
    return xcd * per + (xcd < rem ? xcd : rem) + local;
}

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

// Most tiles of `tile` rows that M rows in `groups` groups and the rows
// behind the last group can need.
int64_t max_tiles(int64_t M, int groups, int tile) {
    const int64_t g = (groups < M ? groups : M) + 1;
    return (M + (tile - 1) * g) / tile;
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

// Workgroups of the largest grid the entry points let through (a grid of
// 512-thread workgroups must stay below 2^32 threads).
constexpr int64_t kMaxBlocks = int64_t(1) << 22;

bool grouped_gemm_fits(int64_t M, int64_t N, int groups) {
    return max_tiles(M, groups, 128) * cdiv(N, 128) < kMaxBlocks;
}

bool grouped_wgrad_fits(int64_t N, int64_t K, int groups) {
    return groups * (cdiv(N, 128) * cdiv(K, 128)) < kMaxBlocks;
}

hipError_t launch_gemm_grouped(const GroupedGemmArgs &a, hipStream_t stream) {
    return a.M >= 128 * (int64_t)a.groups ? launch_shape<MainShape>(a, stream) : launch_shape<TailShape>(a, stream);
}

hipError_t launch_gemm_grouped_wgrad(const GroupedGemmArgs &a, hipStream_t stream) {
    return launch_wgrad_shape<MainShape>(a, stream);
}

}  // namespace mx
