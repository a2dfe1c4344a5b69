// gdn2_rows.h -- device-side building blocks of the norms: rows that a few lanes to a whole workgroup
// hold in registers.
#pragma once

#include "gdn2_device.h"

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

// the largest of values that are not below zero, likewise
template <int LANES>
__device__ __forceinline__ float row_max(float v, float (*scratch)[LANES > 64 ? LANES / 64 : 1], int slot) {
    if constexpr (LANES < 64) {
        v = fmaxf(v, dpp<0x128, 0xf>(v));
        v = fmaxf(v, dpp<0x124, 0xf>(v));
        v = fmaxf(v, dpp<0x122, 0xf>(v));
        v = fmaxf(v, dpp<0x121, 0xf>(v));
        if constexpr (LANES == 32) v = fmaxf(v, __shfl_xor(v, 16));
        return v;
    }
    v = fmaxf(v, dpp<0x111, 0xf>(v));
    v = fmaxf(v, dpp<0x112, 0xf>(v));
    v = fmaxf(v, dpp<0x114, 0xf>(v));
    v = fmaxf(v, dpp<0x118, 0xf>(v));
    v = fmaxf(v, dpp<0x142, 0xa>(v));
    v = fmaxf(v, dpp<0x143, 0xc>(v));
    v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
    if constexpr (LANES > 64) {
        if ((threadIdx.x & 63) == 0) scratch[slot][threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < LANES / 64; ++w) v = fmaxf(v, scratch[slot][w]);
    }
    return v;
}

// A lane's elements of a row: vectors lane, lane + LANES, ... of V.  Rows start at any element
// address; elements behind the row are zeros.
template <typename T, int LANES, int NV, int VEC = 16 / (int)sizeof(T)>
struct Row {
    static constexpr int V = VEC;
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

// lanes of a row and threads of a workgroup, by the row's width (as by_width)
inline int lanes_of(int64_t width) {
    int lanes = 16;
    while (lanes < 1024 && width > lanes * 8) lanes *= 2;
    return lanes;
}
inline int threads_of(int64_t width) { return lanes_of(width) <= 64 ? 256 : lanes_of(width); }

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

}  // namespace norm
}  // namespace gdn2
