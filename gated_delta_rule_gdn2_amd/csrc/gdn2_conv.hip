// gdn2_conv.hip -- the short causal convolution in front of a recurrence, with the inputs that it
// keeps between calls.
//
//   y[t, c] = SiLU(bias[c] + sum_j taps[c, j] x[t - 3 + j, c]),  j = 0 .. 3
//
// Inputs before a sequence's first token are the last three of the call before (the state: row j
// of [3, C] is the input 3 - j tokens ago), or zeros.
#include "gdn2_device.h"
#include "gdn2_launch.h"

namespace gdn2 {
namespace conv {

constexpr int CH = 8;  // channels per thread

// the sequence of a packed token: the last one that starts at or before it (offsets as they
// stand; any offsets give a sequence in [0, n))
__device__ __forceinline__ int sequence_of(const int64_t* __restrict__ cu, int n, int64_t t) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <typename T>
__device__ __forceinline__ Vec<float, CH> load_f32(const T* p) {
    const Vec<T, CH> r = load_vec_any<T, CH>(p);
    Vec<float, CH> f;
#pragma unroll
    for (int e = 0; e < CH; ++e) f.v[e] = to_f32(r.v[e]);
    return f;
}

// the input of a sequence's token t - k, t < start + k: from the state or zero
template <typename T>
__device__ __forceinline__ Vec<float, CH> input_at(const T* __restrict__ x, const T* __restrict__ s0, int64_t seq,
                                                   int64_t start, int64_t t, int64_t C, int64_t xs, int c0) {
    Vec<float, CH> f;
#pragma unroll
    for (int e = 0; e < CH; ++e) f.v[e] = 0.f;
    if (t >= start) return load_f32(x + t * xs + c0);
    if (s0) return load_f32(s0 + (seq * 3 + (3 + t - start)) * C + c0);
    return f;
}

// a thread: one token, eight channels
template <typename T>
__global__ __launch_bounds__(256) void fwd_kernel(const T* __restrict__ x, const float* __restrict__ taps,
                                                  const float* __restrict__ bias, const T* __restrict__ s0,
                                                  T* __restrict__ y, const int64_t* __restrict__ cu, int n, int64_t T_,
                                                  int64_t tokens, int64_t C, int64_t xs) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t nc = C / CH, t = id / nc;
    if (t >= tokens) return;
    const int c0 = (int)(id % nc) * CH;
    int64_t seq, start;
    if (cu) {
        seq = sequence_of(cu, n, t);
        start = min(max(cu[seq], (int64_t)0), tokens);
        if (t < start || t >= cu[seq + 1]) return;  // a token of no sequence
    } else {
        seq = t / T_;
        start = seq * T_;
    }
    float u[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) u[e] = bias ? bias[c0 + e] : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const Vec<float, CH> v = input_at(x, s0, seq, start, t - 3 + j, C, xs, c0);
#pragma unroll
        for (int e = 0; e < CH; ++e) u[e] += taps[(c0 + e) * 4 + j] * v.v[e];
    }
#pragma unroll
    for (int e = 0; e < CH; ++e) y[t * C + c0 + e] = from_f32<T>(u[e] * sigmoid_f(u[e]));
}

// the last three inputs of every sequence
template <typename T>
__global__ __launch_bounds__(256) void state_kernel(const T* __restrict__ x, const T* s0, T* sT,
                                                    const int64_t* __restrict__ cu, int n, int64_t T_, int64_t tokens,
                                                    int64_t C, int64_t xs) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t nc = C / CH, seq = id / nc;
    if (seq >= n) return;
    const int c0 = (int)(id % nc) * CH;
    int64_t start, end;
    if (cu) {
        start = min(max(cu[seq], (int64_t)0), tokens);
        end = min(max(cu[seq + 1], start), tokens);
    } else {
        start = seq * T_;
        end = start + T_;
    }
    Vec<float, CH> v[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) v[j] = input_at(x, s0, seq, start, end - 3 + j, C, xs, c0);
#pragma unroll
    for (int j = 0; j < 3; ++j)
#pragma unroll
        for (int e = 0; e < CH; ++e) sT[(seq * 3 + j) * C + c0 + e] = from_f32<T>(v[j].v[e]);
}

template <typename T>
hipError_t launch(const ConvArgs& a) {
    const int64_t tokens = a.cu_seqlens ? a.T : a.N * a.T;
    const int64_t work = tokens * (a.C / CH), ws = a.N * (a.C / CH);
    if (work > 0)
        hipLaunchKernelGGL((fwd_kernel<T>), dim3((unsigned)((work + 255) / 256)), dim3(256), 0, (hipStream_t)a.stream,
                           (const T*)a.x, a.taps, a.bias, (const T*)a.initial_state, (T*)a.y, a.cu_seqlens, (int)a.N,
                           a.T, tokens, a.C, a.x_stride);
    if (a.final_state)
        hipLaunchKernelGGL((state_kernel<T>), dim3((unsigned)((ws + 255) / 256)), dim3(256), 0, (hipStream_t)a.stream,
                           (const T*)a.x, (const T*)a.initial_state, (T*)a.final_state, a.cu_seqlens, (int)a.N, a.T,
                           tokens, a.C, a.x_stride);
    return hipGetLastError();
}

}  // namespace conv

hipError_t launch_short_conv(const ConvArgs& a) { return a.dtype_bf16 ? conv::launch<bf16>(a) : conv::launch<float>(a); }

// a step is sequences of one token
hipError_t launch_short_conv_step(const ConvArgs& a) { return launch_short_conv(a); }

}  // namespace gdn2
