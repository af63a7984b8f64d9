// The norm of the gradients of many tensors, and gradients scaled by it.
//
//   sum_sq = sum over all tensors of g^2         norm = grad_scale sqrt(sum_sq)
//   scale = grad_scale min(1, max_norm / (norm + 1e-6)),   g = g scale
//
// Squares and sums are in 64 bits: a square of an fp32 gradient neither
// overflows nor vanishes, and the order of a long sum does not show in the fp32
// norm.  The order is fixed all the same: a workgroup sums a chunk of a tensor,
// the sums of the chunks go to the workspace, and one workgroup adds them in
// order; there are no atomics.  Chunks grow with the total so that there are
// about 2048 of them, 8 workgroups a CU; a few short tensors take one launch of
// one workgroup, a wave each.
//
// Bound by memory: the norm reads G, the scaling reads and writes it.  The
// scaling walks the chunks backwards, so that what the norm read last is read
// first.  Measured on MI355X, norm and scaling: 201M fp32 417 us, 5.8 TB/s (463
// with cached instead of non-temporal loads in the norm), 76M bf16 in 40 tensors
// 93 us, 4.9 TB/s (98).  The norm alone, 201M fp32: 123 us, 6.5 TB/s.

#include <cstddef>
#include <cstring>

#include "mx_internal.h"

namespace mx {
namespace {

typedef float f4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
typedef float f2_t __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack(float a, float b) {   // nearest even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2_t{a, b}), bf2_t));
}

__device__ __forceinline__ void add_square(double &s, float v) { s = __builtin_fma((double)v, (double)v, s); }

template <bool F32>
__device__ __forceinline__ void add_squares(double (&s)[2], u4_t v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (F32) {
            add_square(s[e & 1], __uint_as_float(v[e]));
        } else {
            add_square(s[0], low(v[e]));
            add_square(s[1], high(v[e]));
        }
    }
}

// Sum of squares of n elements at p (16-byte aligned) that this lane of
// `lanes` takes.
template <bool F32>
__device__ __forceinline__ double lane_sum(const void *p, int64_t n, int lane, int lanes) {
    constexpr int kPer = F32 ? 4 : 8;   // elements of a 16-byte load
    const u4_t *v = static_cast<const u4_t *>(p);
    const int64_t full = n / kPer;
    double s[2] = {0.0, 0.0};
    int64_t i = lane;
    for (; i + 3 * (int64_t)lanes < full; i += 4 * (int64_t)lanes) {
        u4_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = __builtin_nontemporal_load(v + i + u * (int64_t)lanes);
#pragma unroll
        for (int u = 0; u < 4; ++u) add_squares<F32>(s, w[u]);
    }
    for (; i < full; i += lanes) add_squares<F32>(s, v[i]);
    const int64_t rest = full * kPer + lane;
    if (rest < n) {
        if constexpr (F32) add_square(s[0], static_cast<const float *>(p)[rest]);
        else add_square(s[0], low(static_cast<const uint16_t *>(p)[rest]));
    }
    return s[0] + s[1];
}

__device__ __forceinline__ double wave_sum(double s) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m, 64);
    return s;
}

__device__ __forceinline__ double item_sum(const GradItem &it, int64_t first, int64_t n, int lane, int lanes) {
    return it.f32 ? lane_sum<true>(static_cast<const float *>(it.g) + first, n, lane, lanes)
                  : lane_sum<false>(static_cast<const uint16_t *>(it.g) + first, n, lane, lanes);
}

__device__ __forceinline__ void write_info(double sum_sq, const GradNormOut &o) {
    const double norm = sqrt(sum_sq) * o.grad_scale;
    double part = o.max_norm / (norm + 1e-6);
    part = part > 1.0 || o.max_norm == __builtin_inf() ? 1.0 : part;   // (NaN stays, but where nothing is clipped)
    const float scale = (float)(part * o.grad_scale);
    o.info->sum_sq = sum_sq;
    o.info->norm = (float)norm;
    o.info->scale = scale;
    if (o.step) o.step->grad_scale = scale;
}

// The item of chunk b (chunks counted in this table).
template <int ITEMS>
__device__ __forceinline__ int item_of(const GradTable<ITEMS> &t, uint32_t b) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (b < t.t[mid].chunk_end) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

template <int ITEMS>
__global__ __launch_bounds__(kThreads) void grad_sum_kernel(GradTable<ITEMS> t, double *__restrict__ sums) {
    __shared__ double s_sum[kThreads / 64];
    const int i = item_of(t, blockIdx.x);
    const GradItem &it = t.t[i];
    const int64_t first = (int64_t)(blockIdx.x - (i ? t.t[i - 1].chunk_end : 0u)) * t.chunk;
    const int64_t n = it.numel - first < t.chunk ? it.numel - first : t.chunk;
    const double s = wave_sum(item_sum(it, first, n, threadIdx.x, kThreads));
    if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) sums[blockIdx.x] = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
}

// (1024 threads, so that the loads of 2048 sums are two a lane: 4.7 us with 256)
constexpr int kNormThreads = 1024;
__global__ __launch_bounds__(kNormThreads) void grad_norm_kernel(const double *__restrict__ sums, int n, GradNormOut o) {
    __shared__ double s_sum[kNormThreads / 64];
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kNormThreads) s += sums[i];
    s = wave_sum(s);
    if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x < 64) {
        s = wave_sum(threadIdx.x < kNormThreads / 64 ? s_sum[threadIdx.x] : 0.0);
        if (threadIdx.x == 0) write_info(s, o);
    }
}

__global__ void grad_finish_kernel(GradNormOut o) {
    if (threadIdx.x == 0) write_info(o.info->sum_sq, o);
}

__global__ __launch_bounds__(64 * kGradFew) void grad_norm_few_kernel(GradTable<kGradFew> t, GradNormOut o) {
    __shared__ double s_sum[kGradFew];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    double s = 0.0;
    if (wave < t.count) s = wave_sum(item_sum(t.t[wave], 0, t.t[wave].numel, lane, 64));
    if (lane == 0) s_sum[wave] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kGradFew; ++w) s += s_sum[w];
        write_info(s, o);
    }
}

template <int ITEMS>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(GradTable<ITEMS> t, const mx_grad_norm_info *__restrict__ info) {
    const uint32_t b = gridDim.x - 1 - blockIdx.x;
    const int i = item_of(t, b);
    const GradItem &it = t.t[i];
    const int64_t first = (int64_t)(b - (i ? t.t[i - 1].chunk_end : 0u)) * t.chunk;
    const int64_t n = it.numel - first < t.chunk ? it.numel - first : t.chunk;
    const float scale = info->scale;
    const int per = it.f32 ? 4 : 8;
    u4_t *v = reinterpret_cast<u4_t *>(static_cast<uint8_t *>(it.g) + first * (it.f32 ? 4 : 2));
    const int64_t full = n / per;
    const auto scaled = [&](u4_t w) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = it.f32 ? __float_as_uint(__uint_as_float(w[e]) * scale) : pack(low(w[e]) * scale, high(w[e]) * scale);
        return w;
    };
    int64_t k = threadIdx.x;
    for (; k + 3 * kThreads < full; k += 4 * kThreads) {
        u4_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = v[k + u * kThreads];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[k + u * kThreads] = scaled(w[u]);
    }
    for (; k < full; k += kThreads) v[k] = scaled(v[k]);
    const int64_t rest = full * per + threadIdx.x;
    if (rest < n) {
        if (it.f32) {
            float *p = reinterpret_cast<float *>(v) + rest;
            *p = *p * scale;
        } else {
            uint16_t *p = reinterpret_cast<uint16_t *>(v) + rest;
            *p = (uint16_t)pack(low(*p) * scale, 0.0f);
        }
    }
}

// A few tensors go with a short table, as the arguments are copied for each launch.
template <int ITEMS>
GradTable<ITEMS> short_table(const GradBatch &b) {
    GradTable<ITEMS> t;
    memcpy(&t, &b, offsetof(GradBatch, t) + b.count * sizeof(GradItem));
    return t;
}

}  // namespace

hipError_t launch_grad_sums(const GradBatch &b, double *sums, hipStream_t stream) {
    const dim3 grid(b.t[b.count - 1].chunk_end);
    if (b.count <= kGradFew)
        hipLaunchKernelGGL(grad_sum_kernel<kGradFew>, grid, dim3(kThreads), 0, stream, short_table<kGradFew>(b), sums);
    else
        hipLaunchKernelGGL(grad_sum_kernel<kGradItems>, grid, dim3(kThreads), 0, stream, b, sums);
    return hipGetLastError();
}

hipError_t launch_grad_norm(const double *sums, int n, const GradNormOut &o, hipStream_t stream) {
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kNormThreads), 0, stream, sums, n, o);
    return hipGetLastError();
}

hipError_t launch_grad_norm_few(const GradBatch &b, const GradNormOut &o, hipStream_t stream) {
    hipLaunchKernelGGL(grad_norm_few_kernel, dim3(1), dim3(64 * kGradFew), 0, stream, short_table<kGradFew>(b), o);
    return hipGetLastError();
}

hipError_t launch_grad_finish(const GradNormOut &o, hipStream_t stream) {
    hipLaunchKernelGGL(grad_finish_kernel, dim3(1), dim3(64), 0, stream, o);
    return hipGetLastError();
}

hipError_t launch_grad_scale(const GradBatch &b, const mx_grad_norm_info *info, hipStream_t stream) {
    const dim3 grid(b.t[b.count - 1].chunk_end);
    if (b.count <= kGradFew)
        hipLaunchKernelGGL(grad_scale_kernel<kGradFew>, grid, dim3(kThreads), 0, stream, short_table<kGradFew>(b), info);
    else
        hipLaunchKernelGGL(grad_scale_kernel<kGradItems>, grid, dim3(kThreads), 0, stream, b, info);
    return hipGetLastError();
}

}  // namespace mx
