// gdn2_rotary.hip -- rotary positions on the first channels of the heads of q and k.
//
//   (a, b) -> scale (a cos t - b sin t, a sin t + b cos t),  t = position * frequency of the pair
//
// Pair i of rot / 2 is channels i and i + rot / 2, or 2 i and 2 i + 1 (interleaved); channels from rot
// on are copied.  The inverse turns by -t, which with the same scale is the gradient.
//
// Bound by HBM (each element read and written once), so angles are formed once a token, for all heads
// of q and k, and wait in LDS.  An angle is a product in 64 bits, reduced to a part of a turn there: off by
// 2^-51 of itself, less than fp32's 2^-24 of a turn up to 2^29 radians.  A thread takes the same channels of a head in one
// token after the other.  Where sizes are powers of two a wave's lanes lie side by side in memory and
// exchange the members of their pairs: 8 x 4096 tokens of 24 heads of 128 in bf16, half of each turned,
// take 79 us (5.1 TB/s; a copy of 2 GiB reaches 4.9), against 109 us with both members in one lane.
// Other sizes take 16 bytes of both members a lane where addresses and sizes are whole 16-byte units,
// an element at a time where they are not.
#include "gdn2_device.h"
#include "gdn2_launch.h"

namespace gdn2 {
namespace rotary {

constexpr int kAngles = 2048;  // pairs of all of a workgroup's tokens

// The angles of `count` tokens from t0 on, turn[token][pair]
__device__ __forceinline__ void angles(const RotaryArgs& a, int64_t t0, int count, float2* turn) {
    const int half = (int)a.half;
    for (int i = threadIdx.x; i < count * half; i += blockDim.x) {
        const int64_t t = t0 + i / half;
        const int64_t pos = a.positions ? a.positions[t] : t % a.T;
        const double turns = (double)pos * (double)a.freq[i % half] * 0.15915494309189533577;
        const float part = (float)(turns - rint(turns));
        float s, c;
        sincospif(2.f * part, &s, &c);
        turn[i] = float2{a.scale * c, a.inverse ? -a.scale * s : a.scale * s};
    }
    __syncthreads();
}

// A lane a 16-byte unit of a head, the lanes side by side: loads and stores are whole lines.  The other member of
// a pair of halves comes from the lane half / V away, so units of a head and of a half are powers of two.
template <typename T, int V, bool INTER>
__global__ void units_kernel(RotaryArgs a, int tokens_each, int units, bool in_place) {
    __shared__ float2 turn[kAngles];
    const int half = (int)a.half, heads = (int)a.H, wide = (int)(a.H + a.G) * units, away = half / V;
    const int64_t t0 = (int64_t)blockIdx.x * tokens_each;
    const int count = (int)((a.tokens - t0) < tokens_each ? a.tokens - t0 : tokens_each);
    angles(a, t0, count, turn);
    const int at_once = wide < (int)blockDim.x ? (int)blockDim.x / wide : 1;
    const int sub = wide < (int)blockDim.x ? (int)threadIdx.x / wide : 0;
    if (sub >= at_once) return;
    for (int it = wide < (int)blockDim.x ? (int)threadIdx.x % wide : (int)threadIdx.x; it < wide; it += blockDim.x) {
        const int head = it / units, unit = it % units;
        const bool of_q = head < heads, turned = unit * V < 2 * half;
        const int64_t in_stride = of_q ? a.q_stride : a.k_stride, out_stride = of_q ? a.qo_stride : a.ko_stride;
        const int64_t at = (int64_t)(of_q ? head : head - heads) * a.d + unit * V;
        const T* in = (const T*)(of_q ? a.q : a.k) + at + t0 * in_stride;
        T* out = (T*)(of_q ? a.qo : a.ko) + at + t0 * out_stride;
        const float2* w0 = turn + (INTER ? unit * (V / 2) : unit % (away > 0 ? away : 1) * V);
        const float sign = unit < away ? -1.f : 1.f;
        for (int t = sub; t < count; t += at_once) {
            typedef int i32x4 __attribute__((ext_vector_type(4)));
            i32x4 raw = *reinterpret_cast<const i32x4*>(in + t * in_stride), other = raw;
            if constexpr (!INTER) {
#pragma unroll
                for (int e = 0; e < 4; ++e) other[e] = __shfl_xor(raw[e], away);
            }
            if (turned) {
                const Vec<T, V> x = __builtin_bit_cast(Vec<T, V>, raw), z = __builtin_bit_cast(Vec<T, V>, other);
                const float2* w = w0 + t * half;
                Vec<T, V> y;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 u = w[INTER ? e / 2 : e];
                    if constexpr (INTER)
                        y.v[e] = from_f32<T>(e % 2 ? to_f32(x.v[e - 1]) * u.y + to_f32(x.v[e]) * u.x : to_f32(x.v[e]) * u.x - to_f32(x.v[e + 1]) * u.y);
                    else
                        y.v[e] = from_f32<T>(to_f32(x.v[e]) * u.x + sign * u.y * to_f32(z.v[e]));
                }
                raw = __builtin_bit_cast(i32x4, y);
            }
            if (turned || !in_place) *reinterpret_cast<i32x4*>(out + t * out_stride) = raw;
        }
    }
}

template <typename T, int V, bool INTER>
__global__ void rotary_kernel(RotaryArgs a, int tokens_each, int items, int turned) {
    __shared__ float2 turn[kAngles];
    const int half = (int)a.half, heads = (int)a.H, all = (int)(a.H + a.G);
    const int64_t t0 = (int64_t)blockIdx.x * tokens_each;
    const int count = (int)((a.tokens - t0) < tokens_each ? a.tokens - t0 : tokens_each);
    angles(a, t0, count, turn);
    // items of all heads side by side; several tokens at a time where they are few
    const int wide = all * items, at_once = wide < (int)blockDim.x ? (int)blockDim.x / wide : 1;
    const int sub = wide < (int)blockDim.x ? (int)threadIdx.x / wide : 0;
    if (sub >= at_once) return;
    for (int it = wide < (int)blockDim.x ? (int)threadIdx.x % wide : (int)threadIdx.x; it < wide; it += blockDim.x) {
        const int head = it / items, item = it % items;
        const bool of_q = head < heads;
        const int64_t in_stride = of_q ? a.q_stride : a.k_stride, out_stride = of_q ? a.qo_stride : a.ko_stride;
        const T* in = (const T*)(of_q ? a.q : a.k) + (int64_t)(of_q ? head : head - heads) * a.d + t0 * in_stride;
        T* out = (T*)(of_q ? a.qo : a.ko) + (int64_t)(of_q ? head : head - heads) * a.d + t0 * out_stride;
        if (item >= turned) {  // not rotated
            const int c = 2 * half + (item - turned) * V;
            for (int t = sub; t < count; t += at_once) {
                const Vec<T, V> x = load_vec<T, V>(in + t * in_stride + c);
                float y[V];
#pragma unroll
                for (int e = 0; e < V; ++e) y[e] = to_f32(x.v[e]);
                store_vec_any<T, V>(out + t * out_stride + c, y);
            }
        } else if (INTER && V > 1) {
            const int c = item * V;
#pragma unroll 2
            for (int t = sub; t < count; t += at_once) {
                const Vec<T, V> x = load_vec<T, V>(in + t * in_stride + c);
                const float2* w = turn + t * half + c / 2;
                float y[V];
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    const float2 u = w[e / 2];
                    const float p = to_f32(x.v[e]), q = to_f32(x.v[e + 1]);
                    y[e] = p * u.x - q * u.y;
                    y[e + 1] = p * u.y + q * u.x;
                }
                store_vec_any<T, V>(out + t * out_stride + c, y);
            }
        } else {
            const int c = item * V, first = INTER ? 2 * c : c, second = INTER ? 2 * c + 1 : c + half;
#pragma unroll 2
            for (int t = sub; t < count; t += at_once) {
                const Vec<T, V> x = load_vec<T, V>(in + t * in_stride + first), z = load_vec<T, V>(in + t * in_stride + second);
                const float2* w = turn + t * half + c;
                float y0[V], y1[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 u = w[e];
                    const float p = to_f32(x.v[e]), q = to_f32(z.v[e]);
                    y0[e] = p * u.x - q * u.y;
                    y1[e] = p * u.y + q * u.x;
                }
                store_vec_any<T, V>(out + t * out_stride + first, y0);
                store_vec_any<T, V>(out + t * out_stride + second, y1);
            }
        }
    }
}

// How a call is laid out: whole vectors of 16 bytes, or an element at a time.
struct Plan {
    bool whole, units, in_place;
    int items, turned;  // of a head; of them those that turn
    int64_t each, blocks, threads;
};
Plan plan(const RotaryArgs& a) {
    const int half = (int)a.half, rest = (int)a.d - 2 * half, v = a.dtype_bf16 ? 8 : 4;
    Plan p;
    p.whole = a.d % v == 0 && (a.interleaved ? 2 * half : half) % v == 0;
    for (int64_t s : {a.q_stride, a.qo_stride, a.G ? a.k_stride : 0, a.G ? a.ko_stride : 0}) p.whole = p.whole && s % v == 0;
    for (const void* x : {a.q, (const void*)a.qo, a.k, (const void*)a.ko}) p.whole = p.whole && ((uintptr_t)x & 15) == 0;
    const int V = p.whole ? v : 1;
    p.in_place = a.q == a.qo && a.k == a.ko;
    auto power = [](int64_t n) { return n > 0 && (n & (n - 1)) == 0; };
    p.units = p.whole && power(a.d / v) && a.d / v <= 64 && (a.interleaved || power(half / v));
    p.turned = a.interleaved && V > 1 ? 2 * half / V : half / V;
    p.items = p.units ? (int)a.d / V : p.turned + (p.in_place ? 0 : rest / V);
    // 8 tokens a workgroup, fewer where that leaves the GPU without work
    p.each = a.tokens / 1024;
    p.each = p.each < 1 ? 1 : p.each > 8 ? 8 : p.each;
    if (p.each * half > kAngles) p.each = kAngles / half;
    const int64_t wide = (a.H + a.G) * p.items;
    p.threads = wide >= 1024 ? 1024 : wide > 192 ? (wide + 63) / 64 * 64 : 256;
    p.blocks = (a.tokens + p.each - 1) / p.each;
    return p;
}
template <typename T, int V, bool INTER>
hipError_t run(const RotaryArgs& a, const Plan& p) {
    if (V > 1 && p.units)
        hipLaunchKernelGGL((units_kernel<T, 16 / (int)sizeof(T), INTER>), dim3((unsigned)p.blocks), dim3((unsigned)p.threads), 0, (hipStream_t)a.stream,
                           a, (int)p.each, p.items, p.in_place);
    else
        hipLaunchKernelGGL((rotary_kernel<T, V, INTER>), dim3((unsigned)p.blocks), dim3((unsigned)p.threads), 0, (hipStream_t)a.stream,
                       a, (int)p.each, p.items, p.turned);
    return hipGetLastError();
}
template <typename T>
hipError_t dispatch(const RotaryArgs& a) {
    constexpr int V = 16 / (int)sizeof(T);
    const Plan p = plan(a);
    if (a.interleaved) return p.whole ? run<T, V, true>(a, p) : run<T, 1, true>(a, p);
    return p.whole ? run<T, V, false>(a, p) : run<T, 1, false>(a, p);
}

}  // namespace rotary

bool rotary_grid_ok(const RotaryArgs& a) {
    const rotary::Plan p = rotary::plan(a);
    return p.blocks < ((int64_t)1 << 32) / p.threads;
}

hipError_t launch_rotary(const RotaryArgs& a) {
    return a.dtype_bf16 ? rotary::dispatch<bf16>(a) : rotary::dispatch<float>(a);
}

}  // namespace gdn2
