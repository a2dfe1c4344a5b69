// gdn2_rms.hip -- root-mean-square norm of a residual sum, with an output in the input's type or in 8
// bits, and its gradients.
//
//   h = x + residual,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd gamma
//   8 bits (e4m3): scale = max|y| / 448 of a row (1 for a row of zeros), the output y (448 / max|y|)
//   (max|y| at least 2^-110)
// and with u = h rstd, v = dy gamma:
//   dx = dh + rstd (v - u mean(u v)),  dgamma = sum over rows of dy u.
//
// Rows are held as layer norm holds them: each read once, into the registers of 16 lanes to a whole
// workgroup, the next row's loads in flight behind the present one's sums.  The statistics and y are formed from the sum in
// fp32, before h is rounded to the residual's type; every output is rounded once.
//
// Bound by HBM: 32768 rows of 2048 in bf16, with a residual and 8 bits out 90 us (5.2 TB/s; a copy of 2 GiB 4.9),
// the gradients 104 us (5.15).
#include "gdn2_launch.h"
#include "gdn2_rows.h"

namespace gdn2 {
namespace norm {

constexpr float kE4m3Max = 448.f;
constexpr float kLeastTop = 0x1p-110f;  // below, the scale and its reciprocal would leave fp32's normal range

// vectors of V values, stored as 8 bits each
template <int LANES, int NV, int V, typename F>
__device__ __forceinline__ void store_row_e4m3(uint8_t* p, int lane, int width, F f) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e0 = (lane + LANES * k) * V;
        typedef uint32_t W __attribute__((ext_vector_type(V / 4), aligned(1)));
        W w;
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            const int i = k * V + 4 * q;
            int x = __builtin_amdgcn_cvt_pk_fp8_f32(f(i), f(i + 1), 0, false);
            w[q] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f(i + 2), f(i + 3), x, true);
        }
        if (e0 + V <= width) {
            *reinterpret_cast<W*>(p + e0) = w;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e0 + e < width) p[e0 + e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
        }
    }
}

// T: x (and y, unless E4M3); R: the residual and the sum, which may be one tensor.  Both are walked in vectors of T's 16 bytes.
template <typename T, typename R, bool E4M3, int LANES, int NV>
__global__ __launch_bounds__(kThreads<LANES>) void rms_kernel(const T* __restrict__ x, const R* residual,
                                                              const float* __restrict__ gamma, void* __restrict__ y,
                                                              float* __restrict__ scale, R* h,
                                                              float* __restrict__ rstd, int64_t rows, int width, float eps) {
    typedef Row<T, LANES, NV> RT;
    constexpr int V = RT::V, E = NV * V, RPB = kThreads<LANES> / LANES;
    typedef Row<R, LANES, NV, V> RR;
    __shared__ float scratch[2][LANES > 64 ? LANES / 64 : 1];
    const int lane = threadIdx.x % LANES;
    const float inv = 1.f / (float)width;
    float g[E];
    load_columns<LANES, NV, V>(g, gamma, lane, width);
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LANES;
    const int64_t step = (int64_t)gridDim.x * RPB;
    RT cur, next;
    RR cur_r, next_r;
    if (row < rows) {
        cur.load(x + row * width, lane, width);
        if (residual) cur_r.load(residual + row * width, lane, width);
    }
    for (int n = 0; row < rows; row += step, ++n) {
        if (row + step < rows) {
            next.load(x + (row + step) * width, lane, width);
            if (residual) next_r.load(residual + (row + step) * width, lane, width);
        }
        float v[E], q = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            v[i] = residual ? cur.f(i) + cur_r.f(i) : cur.f(i);
            q += v[i] * v[i];
        }
        if (residual) store_row<R, LANES, NV, V>(h + row * width, lane, width, [&](int i) { return v[i]; });
        const float r = 1.f / sqrtf(row_sum<LANES>(q, scratch, E4M3 ? 0 : n & 1) * inv + eps);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = v[i] * r * g[i];
        if constexpr (E4M3) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) top = fmaxf(top, fabsf(v[i]));
            top = row_max<LANES>(top, scratch, 1);
            if (!(r == r)) top = r;  // a row of NaN has a scale that says so
            if (top < kLeastTop && top > 0.f) top = kLeastTop;
            const float sc = top == 0.f ? 1.f : top * (1.f / kE4m3Max), to = top == 0.f ? 1.f : kE4m3Max / top;
            store_row_e4m3<LANES, NV, V>((uint8_t*)y + row * width, lane, width, [&](int i) { return v[i] * to; });
            if (lane == 0) scale[row] = sc;
        } else {
            store_row<T, LANES, NV, V>((T*)y + row * width, lane, width, [&](int i) { return v[i]; });
        }
        if (rstd && lane == 0) rstd[row] = r;
        cur = next;
        cur_r = next_r;
    }
}

// One pass over dy, h and dh: dx (which may be dh), and the workgroup's part of the sum over rows.
template <typename T, typename R, int LANES, int NV>
__global__ __launch_bounds__(kThreads<LANES>) void rms_bwd_kernel(const T* __restrict__ dy, const R* __restrict__ h,
                                                                  const float* __restrict__ gamma,
                                                                  const float* __restrict__ rstd, const R* dh,
                                                                  R* dx, float* __restrict__ parts,
                                                                  float* __restrict__ dgamma, int64_t rows, int width) {
    typedef Row<T, LANES, NV> RT;
    constexpr int V = RT::V, E = NV * V, RPB = kThreads<LANES> / LANES;
    typedef Row<R, LANES, NV, V> RR;
    __shared__ float scratch[2][LANES > 64 ? LANES / 64 : 1];
    __shared__ float join[RPB > 1 ? LANES * E : 1];
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const float inv = 1.f / (float)width;
    float g[E], dg[E];
    load_columns<LANES, NV, V>(g, gamma, lane, width);
#pragma unroll
    for (int i = 0; i < E; ++i) dg[i] = 0.f;
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + sub;
    for (int n = 0; row < rows; row += step, ++n) {
        RT ry;
        RR rh, rd;
        ry.load(dy + row * width, lane, width);
        rh.load(h + row * width, lane, width);
        if (dh) rd.load(dh + row * width, lane, width);
        const float r = rstd[row];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float d = ry.f(i), u = rh.f(i) * r;
            dg[i] += d * u;
            s += d * g[i] * u;
        }
        s = row_sum<LANES>(s, scratch, n & 1) * inv;
        store_row<R, LANES, NV, V>(dx + row * width, lane, width, [&](int i) {
            const float d = r * (ry.f(i) * g[i] - rh.f(i) * r * s);
            return dh ? rd.f(i) + d : d;
        });
    }
    // the rows of a workgroup one after the other: a fixed order of the sums
    if constexpr (RPB > 1) {
#pragma unroll
        for (int w = 0; w < RPB; ++w) {
            if (sub == w) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    float* p = join + i * LANES + lane;
                    *p = w ? *p + dg[i] : dg[i];
                }
            }
            __syncthreads();
        }
        if (sub == 0) {
#pragma unroll
            for (int i = 0; i < E; ++i) dg[i] = join[i * LANES + lane];
        }
    }
    if (sub == 0)  // one workgroup: its part is the whole
        store_row<float, LANES, NV, V>(gridDim.x == 1 ? dgamma : parts + (int64_t)blockIdx.x * width, lane, width,
                                       [&](int i) { return dg[i]; });
}

// dgamma from the workgroups' parts: 32 columns a workgroup, 32 threads a column
__global__ __launch_bounds__(1024) void rms_join_kernel(const float* __restrict__ parts, float* __restrict__ dgamma, int width,
                                                        int nparts) {
    __shared__ float sum[32][33];
    const int c = threadIdx.x % 32, r = threadIdx.x / 32, col = blockIdx.x * 32 + c;
    float g = 0.f;
    if (col < width) {
#pragma unroll 4
        for (int p = r; p < nparts; p += 32) g += parts[(int64_t)p * width + col];
    }
    sum[r][c] = g;
    __syncthreads();
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) {
        if (r < k) sum[r][c] += sum[r + k][c];
        __syncthreads();
    }
    if (r == 0 && col < width) dgamma[col] = sum[0][c];
}

// Workgroups that stay for many rows, with gamma in registers: the GPU's 2048 waves a quarter
// (8 a SIMD) forward, three quarters of that in the backward pass.
template <int LANES> constexpr int64_t kRmsBlocks = (1 << 19) / kThreads<LANES>;
int64_t rms_parts_limit(int64_t width) { return threads_of(width) == 1024 ? 512 : 3 * (1 << 17) / threads_of(width); }
// few rows go to one workgroup: no parts, and no second launch to join them
int rms_parts_of(int64_t rows, int64_t width) {
    const int64_t rpb = threads_of(width) / lanes_of(width), b = (rows + rpb - 1) / rpb, most = rms_parts_limit(width);
    if (b <= 8) return rows > 0 ? 1 : 0;
    return (int)(b < most ? b : most);
}

template <typename T, typename R, bool E4M3>
struct Rms {
    const RmsArgs& a;
    template <int LANES, int NV>
    hipError_t run() const {
        constexpr int RPB = kThreads<LANES> / LANES;
        const int64_t want = (a.rows + RPB - 1) / RPB, blocks = want < kRmsBlocks<LANES> ? want : kRmsBlocks<LANES>;
        hipLaunchKernelGGL((rms_kernel<T, R, E4M3, LANES, NV>), dim3((unsigned)blocks), dim3(kThreads<LANES>), 0,
                           (hipStream_t)a.stream, (const T*)a.x, (const R*)a.residual, a.gamma, a.y, a.scale, (R*)a.h, a.rstd,
                           a.rows, (int)a.width, a.eps);
        return hipGetLastError();
    }
};
template <typename T, typename R>
struct RmsBwd {
    const RmsBwdArgs& a;
    template <int LANES, int NV>
    hipError_t run() const {
        const int np = rms_parts_of(a.rows, a.width);
        if (np > 0)
            hipLaunchKernelGGL((rms_bwd_kernel<T, R, LANES, NV>), dim3((unsigned)np), dim3(kThreads<LANES>), 0,
                               (hipStream_t)a.stream, (const T*)a.dy, (const R*)a.h, a.gamma, a.rstd, (const R*)a.dh, (R*)a.dx,
                               a.parts, a.dgamma, a.rows, (int)a.width);
        if (np == 1) return hipGetLastError();
        hipLaunchKernelGGL(rms_join_kernel, dim3((unsigned)((a.width + 31) / 32)), dim3(1024), 0, (hipStream_t)a.stream, a.parts,
                           a.dgamma, (int)a.width, np);
        return hipGetLastError();
    }
};

template <typename T, typename R>
hipError_t launch(const RmsArgs& a) {
    return a.scale ? by_width<T>(a.width, Rms<T, R, true>{a}) : by_width<T>(a.width, Rms<T, R, false>{a});
}

}  // namespace norm

hipError_t launch_rms_norm(const RmsArgs& a) {
    if (!a.dtype_bf16) return norm::launch<float, float>(a);
    return a.residual_bf16 ? norm::launch<bf16, bf16>(a) : norm::launch<bf16, float>(a);
}

size_t rms_bwd_workspace_bytes(int64_t rows, int64_t width) {
    const int64_t np = norm::rms_parts_of(rows, width);
    return np > 1 ? (size_t)(np * width * 4) : 0;
}

hipError_t launch_rms_norm_bwd(const RmsBwdArgs& a) {
    if (!a.dtype_bf16) return norm::by_width<float>(a.width, norm::RmsBwd<float, float>{a});
    if (a.residual_bf16) return norm::by_width<bf16>(a.width, norm::RmsBwd<bf16, bf16>{a});
    return norm::by_width<bf16>(a.width, norm::RmsBwd<bf16, float>{a});
}

}  // namespace gdn2
