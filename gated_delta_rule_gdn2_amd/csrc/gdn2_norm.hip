// gdn2_norm.hip -- layer norm, the step in front of a layer's projections, and its gradients.
//
//   mean = sum(x) / width,  rstd = 1 / sqrt(sum((x - mean)^2) / width + eps)
//   y  = (x - mean) rstd gamma + beta
// and with u = (x - mean) rstd, v = dy gamma:
//   dx = rstd (v - mean(v) - u mean(u v)),  dgamma = sum over rows of dy u,  dbeta = sum of dy.
//
// Both passes read each row once, into registers: the variance is a second pass over registers, not
// a difference of sums, so a row far from zero keeps its accuracy.  8 elements a lane (16 above 8192
// columns): a row takes 16 lanes (up to 128 columns) to a wave (512; no barrier), or a workgroup of
// 128 to 1024 threads.  Workgroups stay for many rows, with gamma (and in the backward pass the sums
// over rows) of a lane's columns in registers.  Statistics and sums are fp32; y and dx are rounded once, on the
// store.  Bound by HBM, so what counts is rows in flight: 32768 rows of 2048 in bf16 took 98 us
// forward and 118 us backward at 32 elements a lane, a wave a row, against 62 and 88 us (4.35 and
// 4.59 TB/s; a copy of 4 GB reaches 4.7) at 8.
#include "gdn2_device.h"
#include "gdn2_launch.h"

namespace gdn2 {
namespace norm {

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
}
// The sum of one value per lane, over the wave and in every lane of it: shifts within rows of 16
// lanes, then each row's sum to the rows behind it.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
    v += dpp<0x112, 0xf>(v);
    v += dpp<0x114, 0xf>(v);
    v += dpp<0x118, 0xf>(v);
    v += dpp<0x142, 0xa>(v);  // row_bcast 15 to rows 1 and 3
    v += dpp<0x143, 0xc>(v);  // row_bcast 31 to rows 2 and 3
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// The same over the LANES lanes of a row.  Sums alternate between two slots of scratch, so that one
// barrier a sum is enough.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float (*scratch)[LANES > 64 ? LANES / 64 : 1], int slot) {
    if constexpr (LANES < 64) {
        v += dpp<0x128, 0xf>(v);  // row_ror 8, 4, 2, 1
        v += dpp<0x124, 0xf>(v);
        v += dpp<0x122, 0xf>(v);
        v += dpp<0x121, 0xf>(v);
        if constexpr (LANES == 32) v += __shfl_xor(v, 16);
        return v;
    }
    v = wave_sum(v);
    if constexpr (LANES > 64) {
        if ((threadIdx.x & 63) == 0) scratch[slot][threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < LANES / 64; ++w) v += scratch[slot][w];
    }
    return v;
}

// A lane's elements of a row: vectors lane, lane + LANES, ... of V.  Rows start at any element
// address; elements behind the row are zeros.
template <typename T, int LANES, int NV>
struct Row {
    static constexpr int V = 16 / (int)sizeof(T);
    Vec<T, V> v[NV];
    __device__ __forceinline__ void load(const T* p, int lane, int width) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e0 = (lane + LANES * k) * V;
            if (e0 + V <= width) {
                v[k] = load_vec_any<T, V>(p + e0);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) v[k].v[e] = e0 + e < width ? p[e0 + e] : from_f32<T>(0.f);
            }
        }
    }
    __device__ __forceinline__ float f(int i) const { return to_f32(v[i / V].v[i % V]); }
};
// fp32 values of a lane's columns, vectors of V, stored as T
template <typename T, int LANES, int NV, int V, typename F>
__device__ __forceinline__ void store_row(T* p, int lane, int width, F f) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e0 = (lane + LANES * k) * V;
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = f(k * V + e);
        if (e0 + V <= width) {
            store_vec_any<T, V>(p + e0, o);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e0 + e < width) p[e0 + e] = from_f32<T>(o[e]);
        }
    }
}
template <int LANES, int NV, int V>
__device__ __forceinline__ void load_columns(float (&g)[NV * V], const float* p, int lane, int width) {
#pragma unroll
    for (int i = 0; i < NV * V; ++i) {
        const int c = (lane + LANES * (i / V)) * V + i % V;
        g[i] = p && c < width ? p[c] : 0.f;
    }
}

template <int LANES> constexpr int kThreads = LANES <= 64 ? 256 : LANES;  // whole rows a workgroup

template <typename T, int LANES, int NV>
__global__ __launch_bounds__(kThreads<LANES>) void fwd_kernel(const T* __restrict__ x, const float* __restrict__ gamma,
                                                              const float* __restrict__ beta, T* __restrict__ y,
                                                              float* __restrict__ mean, float* __restrict__ rstd,
                                                              int64_t rows, int width, float eps) {
    typedef Row<T, LANES, NV> R;
    constexpr int E = NV * R::V, RPB = kThreads<LANES> / LANES;  // elements a lane, rows a workgroup
    __shared__ float scratch[2][LANES > 64 ? LANES / 64 : 1];
    const int lane = threadIdx.x % LANES;
    const float inv = 1.f / (float)width;
    float g[E], b[E];
    load_columns<LANES, NV, R::V>(g, gamma, lane, width);
    load_columns<LANES, NV, R::V>(b, beta, lane, width);
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LANES;
    const int64_t step = (int64_t)gridDim.x * RPB;
    R cur, next;
    if (row < rows) cur.load(x + row * width, lane, width);
    for (; row < rows; row += step) {
        if (row + step < rows) next.load(x + (row + step) * width, lane, width);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s += cur.f(i);
        const float m = row_sum<LANES>(s, scratch, 0) * inv;
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const bool in = (lane + LANES * (i / R::V)) * R::V + i % R::V < width;
            const float d = in ? cur.f(i) - m : 0.f;
            q += d * d;
        }
        const float r = 1.f / sqrtf(row_sum<LANES>(q, scratch, 1) * inv + eps);
        store_row<T, LANES, NV, R::V>(y + row * width, lane, width, [&](int i) { return (cur.f(i) - m) * r * g[i] + b[i]; });
        if (mean && lane == 0) {
            mean[row] = m;
            rstd[row] = r;
        }
        cur = next;
    }
}

// One pass over dy and x: dx, and the workgroup's part of the sums over rows.
template <typename T, int LANES, int NV>
__global__ __launch_bounds__(kThreads<LANES>) void bwd_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                                                              const float* __restrict__ gamma,
                                                              const float* __restrict__ mean,
                                                              const float* __restrict__ rstd, T* __restrict__ dx,
                                                              float* __restrict__ parts, float* __restrict__ dgamma,
                                                              float* __restrict__ dbeta, int64_t rows, int width) {
    typedef Row<T, LANES, NV> R;
    constexpr int E = NV * R::V, RPB = kThreads<LANES> / LANES;
    __shared__ float scratch[2][LANES > 64 ? LANES / 64 : 1];
    __shared__ float join[RPB > 1 ? 2 * LANES * E : 1];
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const float inv = 1.f / (float)width;
    float g[E], dg[E], db[E];
    load_columns<LANES, NV, R::V>(g, gamma, lane, width);
#pragma unroll
    for (int i = 0; i < E; ++i) dg[i] = db[i] = 0.f;
    const int64_t step = (int64_t)gridDim.x * RPB;
    for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < rows; row += step) {
        R ry, rx;
        ry.load(dy + row * width, lane, width);
        rx.load(x + row * width, lane, width);
        const float m = mean[row], r = rstd[row];
        float s = 0.f, su = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float d = ry.f(i), u = (rx.f(i) - m) * r, v = d * g[i];
            dg[i] += d * u;
            db[i] += d;
            s += v;
            su += v * u;
        }
        s = row_sum<LANES>(s, scratch, 0) * inv;
        su = row_sum<LANES>(su, scratch, 1) * inv;
        store_row<T, LANES, NV, R::V>(dx + row * width, lane, width, [&](int i) {
            return r * (ry.f(i) * g[i] - s - (rx.f(i) - m) * r * su);
        });
    }
    // the waves of a workgroup one after the other: a fixed order of the sums
    if constexpr (RPB > 1) {
#pragma unroll
        for (int w = 0; w < RPB; ++w) {
            if (sub == w) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    float* p = join + i * 2 * LANES + lane;
                    p[0] = w ? p[0] + dg[i] : dg[i];
                    p[LANES] = w ? p[LANES] + db[i] : db[i];
                }
            }
            __syncthreads();
        }
        if (sub == 0) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                dg[i] = join[i * 2 * LANES + lane];
                db[i] = join[i * 2 * LANES + LANES + lane];
            }
        }
    }
    if (sub == 0) {
        // one workgroup: its part is the whole
        float* pg = gridDim.x == 1 ? dgamma : parts + (int64_t)blockIdx.x * 2 * width;
        float* pb = gridDim.x == 1 ? dbeta : parts + ((int64_t)blockIdx.x * 2 + 1) * width;
        store_row<float, LANES, NV, R::V>(pg, lane, width, [&](int i) { return dg[i]; });
        if (pb) store_row<float, LANES, NV, R::V>(pb, lane, width, [&](int i) { return db[i]; });
    }
}

// dgamma and dbeta from the workgroups' parts: 32 columns a workgroup, 32 threads a column
constexpr int kJoinCols = 32, kJoinRows = 32;
__global__ __launch_bounds__(kJoinCols* kJoinRows) void join_kernel(const float* __restrict__ parts,
                                                                    float* __restrict__ dgamma,
                                                                    float* __restrict__ dbeta, int width, int nparts) {
    __shared__ float sg[kJoinRows][kJoinCols + 1], sb[kJoinRows][kJoinCols + 1];
    const int c = threadIdx.x % kJoinCols, r = threadIdx.x / kJoinCols, col = blockIdx.x * kJoinCols + c;
    float g = 0.f, b = 0.f;
    if (col < width) {
#pragma unroll 4
        for (int p = r; p < nparts; p += kJoinRows) {
            g += parts[(int64_t)(2 * p) * width + col];
            b += parts[(int64_t)(2 * p + 1) * width + col];
        }
    }
    sg[r][c] = g;
    sb[r][c] = b;
    __syncthreads();
#pragma unroll
    for (int h = kJoinRows / 2; h >= 1; h >>= 1) {
        if (r < h) {
            sg[r][c] += sg[r + h][c];
            sb[r][c] += sb[r + h][c];
        }
        __syncthreads();
    }
    if (r == 0 && col < width) {
        dgamma[col] = sg[0][c];
        if (dbeta) dbeta[col] = sb[0][c];
    }
}

// lanes of a row and threads of a workgroup, by the row's width (as by_width)
int lanes_of(int64_t width) {
    int lanes = 16;
    while (lanes < 1024 && width > lanes * 8) lanes *= 2;
    return lanes;
}
int threads_of(int64_t width) { return lanes_of(width) <= 64 ? 256 : lanes_of(width); }
// Workgroups that stay: those that fit the GPU at once by the registers they take, 8 waves a SIMD
// forward and 6 backward (of which workgroups of 16 waves do not fill the last third: two rounds of
// them).  Twice as many lost up to a third (the last ones start late), half as many up to a half.
template <int LANES> constexpr int64_t kFwdBlocks = (1 << 19) / kThreads<LANES>;
int64_t parts_limit(int64_t width) { return threads_of(width) == 1024 ? 512 : 3 * (1 << 17) / threads_of(width); }
// Few rows, up to 8 for each row that a workgroup takes at once, go to one workgroup: its time stays
// below that of a second launch, and there are no parts to join.
int parts_of(int64_t rows, int64_t width) {
    const int64_t rpb = threads_of(width) / lanes_of(width), b = (rows + rpb - 1) / rpb, most = parts_limit(width);
    if (b <= 8) return rows > 0 ? 1 : 0;
    return (int)(b < most ? b : most);
}

// f<LANES, NV> for a row's width
template <typename T, typename F>
hipError_t by_width(int64_t width, F f) {
    constexpr int V = 16 / (int)sizeof(T);
    if (width <= 16 * 8) return f.template run<16, 8 / V>();
    if (width <= 32 * 8) return f.template run<32, 8 / V>();
    if (width <= 64 * 8) return f.template run<64, 8 / V>();
    if (width <= 128 * 8) return f.template run<128, 8 / V>();
    if (width <= 256 * 8) return f.template run<256, 8 / V>();
    if (width <= 512 * 8) return f.template run<512, 8 / V>();
    if (width <= 1024 * 8) return f.template run<1024, 8 / V>();
    return f.template run<1024, 16 / V>();
}

template <typename T>
struct Fwd {
    const NormArgs& a;
    template <int LANES, int NV>
    hipError_t run() const {
        constexpr int RPB = kThreads<LANES> / LANES;
        const int64_t want = (a.rows + RPB - 1) / RPB, blocks = want < kFwdBlocks<LANES> ? want : kFwdBlocks<LANES>;
        hipLaunchKernelGGL((fwd_kernel<T, LANES, NV>), dim3((unsigned)blocks), dim3(kThreads<LANES>), 0,
                           (hipStream_t)a.stream, (const T*)a.x, a.gamma, a.beta, (T*)a.y, a.mean, a.rstd, a.rows,
                           (int)a.width, a.eps);
        return hipGetLastError();
    }
};
template <typename T>
struct Bwd {
    const NormBwdArgs& a;
    template <int LANES, int NV>
    hipError_t run() const {
        const int np = parts_of(a.rows, a.width);
        if (np > 0)
            hipLaunchKernelGGL((bwd_kernel<T, LANES, NV>), dim3((unsigned)np), dim3(kThreads<LANES>), 0,
                               (hipStream_t)a.stream, (const T*)a.dy, (const T*)a.x, a.gamma, a.mean, a.rstd,
                               (T*)a.dx, a.parts, a.dgamma, a.dbeta, a.rows, (int)a.width);
        if (np == 1) return hipGetLastError();
        hipLaunchKernelGGL(join_kernel, dim3((unsigned)((a.width + kJoinCols - 1) / kJoinCols)),
                           dim3(kJoinCols * kJoinRows), 0, (hipStream_t)a.stream, a.parts, a.dgamma, a.dbeta,
                           (int)a.width, np);
        return hipGetLastError();
    }
};

}  // namespace norm

hipError_t launch_layer_norm(const NormArgs& a) {
    return a.dtype_bf16 ? norm::by_width<bf16>(a.width, norm::Fwd<bf16>{a}) : norm::by_width<float>(a.width, norm::Fwd<float>{a});
}

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t width) {
    const int64_t np = norm::parts_of(rows, width);
    return np > 1 ? (size_t)(np * 2 * width * 4) : 0;
}

hipError_t launch_layer_norm_bwd(const NormBwdArgs& a) {
    return a.dtype_bf16 ? norm::by_width<bf16>(a.width, norm::Bwd<bf16>{a}) : norm::by_width<float>(a.width, norm::Bwd<float>{a});
}

}  // namespace gdn2
