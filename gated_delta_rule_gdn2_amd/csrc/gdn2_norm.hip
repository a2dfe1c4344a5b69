// gdn2_norm.hip -- layer norm, the step in front of a layer's projections, and its gradients.
//
//   mean = sum(x) / width,  rstd = 1 / sqrt(sum((x - mean)^2) / width + eps)
//   y  = (x - mean) rstd gamma + beta
// and with u = (x - mean) rstd, v = dy gamma:
//   dx = rstd (v - mean(v) - u mean(u v)),  dgamma = sum over rows of dy u,  dbeta = sum of dy.
//
// Statistics and sums are fp32; y and dx are rounded once, on the store.
#include "gdn2_device.h"
#include "gdn2_launch.h"

namespace gdn2 {
namespace norm {

constexpr int kThreads = 256;

// the sum of one value per thread, over the workgroup; scratch holds a float per wave
__device__ __forceinline__ float block_sum(float x, float* scratch) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) x += scratch[w];
    return x;
}

// one workgroup a row
template <typename T>
__global__ __launch_bounds__(kThreads) void fwd_kernel(const T* __restrict__ x, const float* __restrict__ gamma,
                                                       const float* __restrict__ beta, T* __restrict__ y,
                                                       float* __restrict__ mean, float* __restrict__ rstd, int width,
                                                       float eps) {
    __shared__ float scratch[kThreads / 64];
    const int64_t row = blockIdx.x;
    const T* xr = x + row * width;
    float s = 0.f;
    for (int i = threadIdx.x; i < width; i += kThreads) s += to_f32(xr[i]);
    const float m = block_sum(s, scratch) / (float)width;
    float q = 0.f;
    for (int i = threadIdx.x; i < width; i += kThreads) {
        const float d = to_f32(xr[i]) - m;
        q += d * d;
    }
    const float r = 1.f / sqrtf(block_sum(q, scratch) / (float)width + eps);
    for (int i = threadIdx.x; i < width; i += kThreads) {
        const float v = (to_f32(xr[i]) - m) * r * gamma[i];
        y[row * width + i] = from_f32<T>(beta ? v + beta[i] : v);
    }
    if (mean && threadIdx.x == 0) {
        mean[row] = m;
        rstd[row] = r;
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dx_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                                                      const float* __restrict__ gamma, const float* __restrict__ mean,
                                                      const float* __restrict__ rstd, T* __restrict__ dx, int width) {
    __shared__ float scratch[kThreads / 64];
    const int64_t row = blockIdx.x;
    const float m = mean[row], r = rstd[row];
    float s = 0.f, su = 0.f;
    for (int i = threadIdx.x; i < width; i += kThreads) {
        const float v = to_f32(dy[row * width + i]) * gamma[i];
        s += v;
        su += v * (to_f32(x[row * width + i]) - m) * r;
    }
    s = block_sum(s, scratch) / (float)width;
    su = block_sum(su, scratch) / (float)width;
    for (int i = threadIdx.x; i < width; i += kThreads) {
        const float v = to_f32(dy[row * width + i]) * gamma[i];
        dx[row * width + i] = from_f32<T>(r * (v - s - (to_f32(x[row * width + i]) - m) * r * su));
    }
}

// dgamma and dbeta over a run of rows: a thread owns a column
template <typename T>
__global__ __launch_bounds__(64) void parts_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                                                   const float* __restrict__ mean, const float* __restrict__ rstd,
                                                   float* __restrict__ parts, int64_t rows, int width, int run) {
    const int col = blockIdx.x * 64 + threadIdx.x;
    if (col >= width) return;
    const int64_t lo = (int64_t)blockIdx.y * run, hi = min(lo + run, rows);
    float g = 0.f, b = 0.f;
    for (int64_t r = lo; r < hi; ++r) {
        const float d = to_f32(dy[r * width + col]);
        g += d * (to_f32(x[r * width + col]) - mean[r]) * rstd[r];
        b += d;
    }
    parts[(int64_t)(2 * blockIdx.y) * width + col] = g;
    parts[(int64_t)(2 * blockIdx.y + 1) * width + col] = b;
}

__global__ __launch_bounds__(64) void join_kernel(const float* __restrict__ parts, float* __restrict__ dgamma,
                                                  float* __restrict__ dbeta, int width, int nparts) {
    const int col = blockIdx.x * 64 + threadIdx.x;
    if (col >= width) return;
    float g = 0.f, b = 0.f;
    for (int p = 0; p < nparts; ++p) {
        g += parts[(int64_t)(2 * p) * width + col];
        b += parts[(int64_t)(2 * p + 1) * width + col];
    }
    dgamma[col] = g;
    if (dbeta) dbeta[col] = b;
}

constexpr int kRun = 128;  // rows of one partial sum
int parts_of(int64_t rows) { return (int)((rows + kRun - 1) / kRun); }

template <typename T>
hipError_t launch_fwd(const NormArgs& a) {
    hipLaunchKernelGGL((fwd_kernel<T>), dim3((unsigned)a.rows), dim3(kThreads), 0, (hipStream_t)a.stream, (const T*)a.x,
                       a.gamma, a.beta, (T*)a.y, a.mean, a.rstd, (int)a.width, a.eps);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_bwd(const NormBwdArgs& a) {
    const int np = parts_of(a.rows);
    const unsigned nc = (unsigned)((a.width + 63) / 64);
    if (a.rows > 0) {
        hipLaunchKernelGGL((dx_kernel<T>), dim3((unsigned)a.rows), dim3(kThreads), 0, (hipStream_t)a.stream,
                           (const T*)a.dy, (const T*)a.x, a.gamma, a.mean, a.rstd, (T*)a.dx, (int)a.width);
        hipLaunchKernelGGL((parts_kernel<T>), dim3(nc, np), dim3(64), 0, (hipStream_t)a.stream, (const T*)a.dy,
                           (const T*)a.x, a.mean, a.rstd, a.parts, a.rows, (int)a.width, kRun);
    }
    hipLaunchKernelGGL(join_kernel, dim3(nc), dim3(64), 0, (hipStream_t)a.stream, a.parts, a.dgamma, a.dbeta,
                       (int)a.width, np);
    return hipGetLastError();
}

}  // namespace norm

hipError_t launch_layer_norm(const NormArgs& a) { return a.dtype_bf16 ? norm::launch_fwd<bf16>(a) : norm::launch_fwd<float>(a); }

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t width) { return (size_t)norm::parts_of(rows) * 2 * width * 4; }

hipError_t launch_layer_norm_bwd(const NormBwdArgs& a) {
    return a.dtype_bf16 ? norm::launch_bwd<bf16>(a) : norm::launch_bwd<float>(a);
}

}  // namespace gdn2
