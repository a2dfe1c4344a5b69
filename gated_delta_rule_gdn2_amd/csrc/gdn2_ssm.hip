// gdn2_ssm.hip -- the selective state space scan over prompts, and its step for single tokens.
//
// Per sequence and head, with a state S of dk rows and dv columns:
//   dt_t = softplus(raw_t + bias),  S_t = exp(dt_t A) S_{t-1} + dt_t B_t x_t^T,
//   y_t = S_t^T C_t + D x_t
// B and C belong to a group of heads.  The columns of S are independent.
#include "gdn2_device.h"
#include "gdn2_launch.h"

namespace gdn2 {
namespace ssm {

// raw + bias, through softplus where asked: max(v, 0) + log(1 + e^-|v|)
__device__ __forceinline__ float time_step(float v, bool softplus) {
    return softplus ? fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))) : v;
}

// A workgroup walks 64 columns of one (sequence, head) token by token; wave w holds a quarter of
// the rows, a lane one column of them.
template <typename T, int DK>
__global__ __launch_bounds__(256) void walk_kernel(const T* __restrict__ x, const T* __restrict__ dt,
                                                   const T* __restrict__ bm, const T* __restrict__ cm,
                                                   const float* __restrict__ A, const float* __restrict__ D,
                                                   const float* __restrict__ dt_bias, const float* s0,
                                                   T* __restrict__ y, float* sT, const int64_t* __restrict__ cu,
                                                   int64_t T_, int H, int G, int dv, int64_t xs, int64_t dts,
                                                   int64_t bs, int64_t cs, bool softplus) {
    constexpr int R = DK / 4;
    __shared__ float part[2][4][64];
    const int slices = dv / 64, slice = blockIdx.x % slices;
    const int h = (blockIdx.x / slices) % H, n = blockIdx.x / slices / H;
    const int g = h / (H / G), w = threadIdx.x >> 6, lane = threadIdx.x & 63, p = slice * 64 + lane;
    int64_t lo = n * T_, hi = lo + T_;
    if (cu) {
        lo = min(max(cu[n], (int64_t)0), T_);
        hi = min(max(cu[n + 1], lo), T_);
    }
    float s[R];
    const int64_t base = (((int64_t)n * H + h) * DK + w * R) * dv + p;
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = s0 ? s0[base + (int64_t)r * dv] : 0.f;
    const float a = A[h], d = D ? D[h] : 0.f, bias = dt_bias ? dt_bias[h] : 0.f;
    for (int64_t t = lo; t < hi; ++t) {
        const float step = time_step(to_f32(dt[t * dts + h]) + bias, softplus);
        const float xv = to_f32(x[t * xs + h * dv + p]), dx = step * xv, decay = expf(step * a);
        const T* br = bm + t * bs + g * DK + w * R;
        const T* cr = cm + t * cs + g * DK + w * R;
        float acc = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] = s[r] * decay + to_f32(br[r]) * dx;
            acc += s[r] * to_f32(cr[r]);
        }
        const int k = (int)(t - lo) & 1;  // one barrier a token: the other half is still being read
        part[k][w][lane] = acc;
        __syncthreads();
        if (w == 0)
            y[(t * H + h) * dv + p] = from_f32<T>(part[k][0][lane] + part[k][1][lane] + part[k][2][lane] + part[k][3][lane] + d * xv);
    }
    if (sT) {
#pragma unroll
        for (int r = 0; r < R; ++r) sT[base + (int64_t)r * dv] = s[r];
    }
}

template <typename T, int DK>
hipError_t launch_walk(const SsmArgs& a) {
    hipLaunchKernelGGL((walk_kernel<T, DK>), dim3((unsigned)(a.N * a.H * (a.dv / 64))), dim3(256), 0,
                       (hipStream_t)a.stream, (const T*)a.x, (const T*)a.dt, (const T*)a.b, (const T*)a.c, a.A, a.D,
                       a.dt_bias, a.initial_state, (T*)a.y, a.final_state, a.cu_seqlens, a.T, (int)a.H, (int)a.G,
                       (int)a.dv, a.x_stride, a.dt_stride, a.b_stride, a.c_stride, a.softplus);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const SsmArgs& a) {
    return a.dk == 128 ? launch_walk<T, 128>(a) : launch_walk<T, 64>(a);
}

}  // namespace ssm

size_t ssm_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, bool, int64_t) { return 0; }

hipError_t launch_ssm_fwd(const SsmArgs& a, void*) {
    return a.dtype_bf16 ? ssm::launch_t<bf16>(a) : ssm::launch_t<float>(a);
}

// a step is sequences of one token, the state first and final
hipError_t launch_ssm_step(const SsmArgs& a) { return launch_ssm_fwd(a, nullptr); }

}  // namespace gdn2
