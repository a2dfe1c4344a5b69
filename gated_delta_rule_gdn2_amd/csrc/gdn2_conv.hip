// gdn2_conv.hip -- the short causal convolution in front of a recurrence, with the inputs that it
// keeps between calls.
//
//   y[t, c] = SiLU(bias[c] + sum_j taps[c, j] x[t - 3 + j, c]),  j = 0 .. 3
//
// Inputs before a sequence's first token are the last three of the call before (the state: row j
// of [3, C] is the input 3 - j tokens ago), or zeros.
//
// A thread takes four channels over a run of consecutive tokens, its taps and the last three
// inputs in registers, so an input is read once but for three rows a run.  Bound by HBM.
#include "gdn2_device.h"
#include "gdn2_launch.h"

namespace gdn2 {
namespace conv {

// Channels a thread.  In bf16 eight, with 16-byte accesses, held 134 registers and took 82 us where
// four take 66 (8 x 4096 tokens of 2304 channels; 4.6 TB/s, the rate of a large copy).
constexpr int CH = 4;

struct Params {
    const void* x;
    const float* taps;
    const float* bias;
    const void* s0;
    void* y;
    void* sT;
    const int64_t* cu;
    int64_t T, tokens, C, xs;  // T: tokens of a sequence (without cu); tokens: of all
    int N, nc;                 // sequences; threads across the channels
    int64_t runs, seq_runs;    // runs of tokens in all, and of a sequence (without cu)
    int64_t run_groups;        // workgroups that walk runs; those behind them form the states
};

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

// A sequence's input of token t, from three before its start on: of the state, or zero.
template <typename T>
__device__ __forceinline__ Vec<T, CH> input_at(const Params& a, int64_t seq, int64_t start, int64_t t, int c0) {
    if (t >= start) return load_vec_any<T, CH>((const T*)a.x + t * a.xs + c0);
    if (a.s0) return load_vec<T, CH>((const T*)a.s0 + (seq * 3 + (3 + t - start)) * a.C + c0);
    Vec<T, CH> z;
#pragma unroll
    for (int e = 0; e < CH; ++e) z.v[e] = from_f32<T>(0.f);
    return z;
}

template <typename T>
__device__ __forceinline__ void put(T* p, const Vec<T, CH>& v) {
    typedef T V __attribute__((ext_vector_type(CH)));
    V x;
#pragma unroll
    for (int e = 0; e < CH; ++e) x[e] = v.v[e];
    *reinterpret_cast<V*>(p) = x;
}

template <typename T>
struct Taps {
    float t[CH][4], b[CH];
    __device__ __forceinline__ void load(const Params& a, int c0) {
#pragma unroll
        for (int e = 0; e < CH; ++e) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(a.taps + (int64_t)(c0 + e) * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) t[e][j] = v[j];
            b[e] = a.bias ? a.bias[c0 + e] : 0.f;
        }
    }
    // y of the inputs w0, w1, w2 before and x
    __device__ __forceinline__ void apply(T* y, const Vec<T, CH>& w0, const Vec<T, CH>& w1, const Vec<T, CH>& w2,
                                          const Vec<T, CH>& x) const {
        Vec<T, CH> o;
#pragma unroll
        for (int e = 0; e < CH; ++e) {
            const float u = b[e] + t[e][0] * to_f32(w0.v[e]) + t[e][1] * to_f32(w1.v[e]) + t[e][2] * to_f32(w2.v[e]) +
                            t[e][3] * to_f32(x.v[e]);
            o.v[e] = from_f32<T>(u * sigmoid_f(u));
        }
        put(y, o);
    }
};

// item `id` of a grid of rows of nc: its row and place, with one wide division a workgroup
__device__ __forceinline__ void place(int64_t first, int nc, int64_t* row, int* col) {
    const int64_t r = first / nc;
    const unsigned c = (unsigned)(first - r * nc) + threadIdx.x;
    *row = r + c / (unsigned)nc;
    *col = (int)(c % (unsigned)nc);
}

template <typename T, int RUN>
__global__ __launch_bounds__(256) void fwd_kernel(Params a) {
    int64_t row;
    int c0;
    if (blockIdx.x >= a.run_groups) {  // a sequence's last three inputs
        place(((int64_t)blockIdx.x - a.run_groups) * 256, a.nc, &row, &c0);
        if (row >= a.N) return;
        c0 *= CH;
        int64_t start = row * a.T, end = start + a.T;
        if (a.cu) {
            start = min(max(a.cu[row], (int64_t)0), a.tokens);
            end = min(max(a.cu[row + 1], start), a.tokens);
        }
        Vec<T, CH> v[3];  // all before the first store: the state may be updated in place
#pragma unroll
        for (int j = 0; j < 3; ++j) v[j] = input_at<T>(a, row, start, end - 3 + j, c0);
#pragma unroll
        for (int j = 0; j < 3; ++j) put((T*)a.sT + (row * 3 + j) * a.C + c0, v[j]);
        return;
    }
    place((int64_t)blockIdx.x * 256, a.nc, &row, &c0);
    if (row >= a.runs) return;
    c0 *= CH;
    Taps<T> taps;
    taps.load(a, c0);
    int64_t seq = 0, start = 0, t = row * RUN, last = min(t + RUN, a.tokens), end = a.tokens;
    if (!a.cu) {
        seq = row / a.seq_runs;
        start = seq * a.T;
        end = start + a.T;
        t = start + (row - seq * a.seq_runs) * RUN;
        last = min(t + RUN, end);
    }
    while (t < last) {
        if (a.cu) {
            seq = sequence_of(a.cu, a.N, t);
            start = min(max(a.cu[seq], (int64_t)0), a.tokens);
            end = min(max(a.cu[seq + 1], start), a.tokens);
            if (t < start) {  // tokens before the first sequence
                t = start;
                continue;
            }
            if (t >= end) {  // behind the last one, or where offsets decrease
                if (seq + 1 >= a.N) return;
                ++t;
                continue;
            }
        }
        const int64_t stop = min(last, end);
        const T* px = (const T*)a.x + c0;
        T* py = (T*)a.y + c0;
        Vec<T, CH> w0 = input_at<T>(a, seq, start, t - 3, c0), w1 = input_at<T>(a, seq, start, t - 2, c0);
        Vec<T, CH> w2 = input_at<T>(a, seq, start, t - 1, c0);
        Vec<T, CH> v[4], next[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = load_vec_any<T, CH>(px + min(t + j, stop - 1) * a.xs);
        while (t < stop) {  // four tokens, the next four's loads before their stores
#pragma unroll
            for (int j = 0; j < 4; ++j) next[j] = load_vec_any<T, CH>(px + min(t + 4 + j, stop - 1) * a.xs);
            taps.apply(py + t * a.C, w0, w1, w2, v[0]);
            if (t + 1 < stop) taps.apply(py + (t + 1) * a.C, w1, w2, v[0], v[1]);
            if (t + 2 < stop) taps.apply(py + (t + 2) * a.C, w2, v[0], v[1], v[2]);
            if (t + 3 < stop) taps.apply(py + (t + 3) * a.C, v[0], v[1], v[2], v[3]);
            w0 = v[1];
            w1 = v[2];
            w2 = v[3];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = next[j];
            t += 4;
        }
        t = stop;
    }
}

// One token: y, and the state moved on by it.
template <typename T>
__global__ __launch_bounds__(256) void step_kernel(Params a) {
    int64_t n;
    int c0;
    place((int64_t)blockIdx.x * 256, a.nc, &n, &c0);
    if (n >= a.N) return;
    c0 *= CH;
    T* st = (T*)a.sT + n * 3 * a.C + c0;
    const Vec<T, CH> w0 = load_vec<T, CH>(st), w1 = load_vec<T, CH>(st + a.C), w2 = load_vec<T, CH>(st + 2 * a.C);
    const Vec<T, CH> x = load_vec_any<T, CH>((const T*)a.x + n * a.xs + c0);
    Taps<T> taps;
    taps.load(a, c0);
    put(st, w1);
    put(st + a.C, w2);
    put(st + 2 * a.C, x);
    taps.apply((T*)a.y + n * a.C + c0, w0, w1, w2, x);
}

template <typename T>
Params params(const ConvArgs& a) {
    return Params{a.x, a.taps, a.bias, a.initial_state, a.y, a.final_state, a.cu_seqlens, a.T,
                  a.cu_seqlens ? a.T : a.N * a.T, a.C, a.x_stride, (int)a.N, (int)(a.C / CH), 0, 0, 0};
}

template <typename T, int RUN>
hipError_t launch_runs(const ConvArgs& a) {
    Params p = params<T>(a);
    p.seq_runs = (a.T + RUN - 1) / RUN;
    p.runs = a.cu_seqlens ? p.seq_runs : p.seq_runs * a.N;
    const int64_t groups = (p.runs * p.nc + 255) / 256, states = a.final_state ? (a.N * p.nc + 255) / 256 : 0;
    // in place, the states are formed by a launch of their own: the runs read the old ones
    const bool apart = states && a.initial_state == a.final_state;
    p.run_groups = groups;
    if (groups + (apart ? 0 : states) > 0)
        hipLaunchKernelGGL((fwd_kernel<T, RUN>), dim3((unsigned)(groups + (apart ? 0 : states))), dim3(256), 0,
                           (hipStream_t)a.stream, p);
    if (apart) {
        p.run_groups = 0;
        hipLaunchKernelGGL((fwd_kernel<T, RUN>), dim3((unsigned)states), dim3(256), 0, (hipStream_t)a.stream, p);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t launch(const ConvArgs& a) {
    // runs of 16 tokens where those fill the GPU, else of 4: more threads, each with less to wait for
    const int64_t tokens = a.cu_seqlens ? a.T : a.N * a.T, threads = tokens / 16 * (a.C / CH);
    return threads >= (1 << 17) ? launch_runs<T, 16>(a) : launch_runs<T, 4>(a);
}

template <typename T>
hipError_t launch_step(const ConvArgs& a) {
    const Params p = params<T>(a);
    hipLaunchKernelGGL((step_kernel<T>), dim3((unsigned)((a.N * p.nc + 255) / 256)), dim3(256), 0,
                       (hipStream_t)a.stream, p);
    return hipGetLastError();
}

}  // namespace conv

hipError_t launch_short_conv(const ConvArgs& a) { return a.dtype_bf16 ? conv::launch<bf16>(a) : conv::launch<float>(a); }

hipError_t launch_short_conv_step(const ConvArgs& a) {
    return a.dtype_bf16 ? conv::launch_step<bf16>(a) : conv::launch_step<float>(a);
}

}  // namespace gdn2
