// gdn2_api_block.hip -- the C ABI of the state space block (include/gdn2.h): the scan, the short
// convolution and layer norm.  Argument validation and dispatch, on the host; nothing is enqueued
// before every check has passed.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/gdn2.h"
#include "gdn2_check.h"
#include "gdn2_launch.h"

namespace {

using gdn2::aligned_to;
using gdn2::mul_ok;
using gdn2::overlap;
using gdn2::Range;
using gdn2::range_of;

constexpr int64_t kMaxStride = int64_t(1) << 22;  // elements between tokens: 64 of them stay below 2^30 bytes
constexpr int64_t kMaxStepStride = int64_t(1) << 31;  // and between a step's, which are multiplied in 64 bits
constexpr int64_t kMaxWidth = 16384;
// Tokens of a sequence, or of all packed ones: indexes a few chunks behind the last stay 32-bit.
constexpr int64_t kMaxTokens = INT_MAX - 1024;
// Sequence-heads: workgroups of 256 threads, of which a launch may have less than 2^32; packed
// sequences that are cut have more pieces than there are sequences.
constexpr int64_t kMaxHeads = INT_MAX / 256;

int64_t elem(gdn2_dtype_t t) { return t == GDN2_DTYPE_BF16 ? 2 : 4; }
bool known(gdn2_dtype_t t) { return t == GDN2_DTYPE_BF16 || t == GDN2_DTYPE_F32; }

// bytes from a strided tensor's first token to the end of its last
bool span(int64_t tokens, int64_t stride, int64_t per_token, int64_t es, int64_t* out) {
    if (tokens <= 0) {
        *out = 0;
        return tokens == 0;
    }
    int64_t e;
    if (!mul_ok(tokens - 1, stride, &e) || e > INT64_MAX / 8 - per_token) return false;
    *out = (e + per_token) * es;
    return true;
}

int device_cus() {
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess) return -1;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return -1;
    return cus;
}

// The scan's checks, for prompts, packed prompts and single tokens.  `tokens` rows in all.
gdn2_status_t check_ssm(const gdn2::SsmArgs& a, gdn2_dtype_t dtype, int64_t tokens, bool in_place) {
    if (!known(dtype)) return GDN2_ERR_UNSUPPORTED;
    if (a.N < 1 || a.T < 0 || tokens < 0 || a.H < 1 || a.G < 1 || a.dk < 1 || a.dv < 1) return GDN2_ERR_SHAPE;
    if (tokens > 0 && (!a.x || !a.dt || !a.b || !a.c || !a.y)) return GDN2_ERR_NULL;
    if (!a.A || (in_place && !a.final_state)) return GDN2_ERR_NULL;
    if (!gdn2::ssm_supported(a.dk, a.dv, dtype == GDN2_DTYPE_BF16, dtype == GDN2_DTYPE_F32)) return GDN2_ERR_UNSUPPORTED;
    if (a.N > INT_MAX || a.T > kMaxTokens || a.H >= kMaxStride || a.H % a.G) return GDN2_ERR_SHAPE;
    if (a.H * a.dv >= kMaxStride || a.G * a.dk >= kMaxStride) return GDN2_ERR_SHAPE;
    if (a.x_stride < a.H * a.dv || a.dt_stride < a.H || a.b_stride < a.G * a.dk || a.c_stride < a.G * a.dk)
        return GDN2_ERR_SHAPE;
    const int64_t far = in_place ? kMaxStepStride : kMaxStride;
    if (a.x_stride >= far || a.dt_stride >= far || a.b_stride >= far || a.c_stride >= far) return GDN2_ERR_SHAPE;
    const int64_t es = elem(dtype);
    int64_t nh, ns, nx, nt, nb, nc, ny;
    if (!mul_ok(a.N, a.H, &nh) || nh > kMaxHeads || !mul_ok(nh, a.dk * a.dv * 4, &ns)) return GDN2_ERR_SHAPE;
    if (!span(tokens, a.x_stride, a.H * a.dv, es, &nx) || !span(tokens, a.dt_stride, a.H, es, &nt) ||
        !span(tokens, a.b_stride, a.G * a.dk, es, &nb) || !span(tokens, a.c_stride, a.G * a.dk, es, &nc) ||
        !span(tokens, a.H * a.dv, a.H * a.dv, es, &ny))
        return GDN2_ERR_SHAPE;
    if ((a.x_stride * es | a.b_stride * es | a.c_stride * es) & 15) return GDN2_ERR_MISALIGNED;
    for (const void* p : {a.x, a.b, a.c, (const void*)a.y, (const void*)a.initial_state, (const void*)a.final_state})
        if (p && !aligned_to(p, 16)) return GDN2_ERR_MISALIGNED;
    for (const float* p : {a.A, a.D, a.dt_bias})
        if (p && !aligned_to(p, 4)) return GDN2_ERR_MISALIGNED;
    if (a.dt && !aligned_to(a.dt, es)) return GDN2_ERR_MISALIGNED;
    const Range ry = range_of(a.y, ny), rf = range_of(a.final_state, a.final_state ? ns : 0);
    const Range rc = range_of(a.cu_seqlens, a.cu_seqlens ? (a.N + 1) * 8 : 0);
    for (const Range& r : {range_of(a.x, nx), range_of(a.dt, nt), range_of(a.b, nb), range_of(a.c, nc), rc,
                           range_of(a.A, a.H * 4), range_of(a.D, a.D ? a.H * 4 : 0),
                           range_of(a.dt_bias, a.dt_bias ? a.H * 4 : 0)})
        if (overlap(ry, r) || overlap(rf, r)) return GDN2_ERR_ALIAS;
    const Range ri = range_of(a.initial_state, a.initial_state ? ns : 0);
    if (overlap(ry, rf) || overlap(ry, ri)) return GDN2_ERR_ALIAS;
    if (a.initial_state != a.final_state && overlap(ri, rf)) return GDN2_ERR_ALIAS;
    return GDN2_OK;
}

size_t ssm_workspace(bool packed, int64_t N, int64_t T, int64_t H, int64_t dk, int64_t dv, gdn2_dtype_t dtype) {
    if (N < 1 || T < 1 || H < 1 || N > INT_MAX || T > kMaxTokens || H > INT_MAX || N * H > kMaxHeads) return 0;
    if (!gdn2::ssm_supported(dk, dv, dtype == GDN2_DTYPE_BF16, dtype == GDN2_DTYPE_F32)) return 0;
    const int cus = device_cus();
    return gdn2::ssm_workspace_bytes(packed, N, T, H, dk, dv, dtype == GDN2_DTYPE_BF16, cus > 0 ? cus : 256);
}

// the scan of whole or packed prompts, with `tokens` rows in all
gdn2_status_t ssm_fwd(gdn2::SsmArgs a, gdn2_dtype_t dtype, int64_t tokens, void* workspace, size_t workspace_bytes) {
    const gdn2_status_t st = check_ssm(a, dtype, tokens, false);
    if (st != GDN2_OK) return st;
    if (workspace || workspace_bytes) {
        const size_t need = ssm_workspace(a.cu_seqlens != nullptr, a.N, a.T, a.H, a.dk, a.dv, dtype);
        if (need == 0 || !workspace || workspace_bytes < need) return GDN2_ERR_WORKSPACE;
        if (!aligned_to(workspace, 256)) return GDN2_ERR_MISALIGNED;
        const int64_t es = elem(dtype), nt = tokens - 1, ns = a.N * a.H * a.dk * a.dv * 4;
        const Range rw = range_of(workspace, (int64_t)need);
        for (const Range& r :
             {range_of(a.x, (nt * a.x_stride + a.H * a.dv) * es), range_of(a.dt, (nt * a.dt_stride + a.H) * es),
              range_of(a.b, (nt * a.b_stride + a.G * a.dk) * es), range_of(a.c, (nt * a.c_stride + a.G * a.dk) * es),
              range_of(a.A, a.H * 4), range_of(a.D, a.D ? a.H * 4 : 0), range_of(a.dt_bias, a.dt_bias ? a.H * 4 : 0),
              range_of(a.initial_state, a.initial_state ? ns : 0), range_of(a.final_state, a.final_state ? ns : 0),
              range_of(a.y, tokens * a.H * a.dv * es), range_of(a.cu_seqlens, a.cu_seqlens ? (a.N + 1) * 8 : 0)})
            if (overlap(rw, r)) return GDN2_ERR_ALIAS;
    }
    if (tokens == 0 && !a.final_state) return GDN2_OK;  // nothing to write
    a.cus = device_cus();
    if (a.cus <= 0) return GDN2_ERR_HIP;
    return gdn2::launch_ssm_fwd(a, workspace) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status_t check_conv(const gdn2::ConvArgs& a, gdn2_dtype_t dtype, int64_t tokens, bool in_place) {
    if (!known(dtype)) return GDN2_ERR_UNSUPPORTED;
    if (a.N < 1 || a.T < 0 || tokens < 0 || a.C < 1 || a.C % 8) return GDN2_ERR_SHAPE;
    if (tokens > 0 && (!a.x || !a.y)) return GDN2_ERR_NULL;
    if (!a.taps || (in_place && !a.final_state)) return GDN2_ERR_NULL;
    const int64_t far = in_place ? kMaxStepStride : kMaxStride;
    if (a.N > INT_MAX || a.T > INT_MAX || a.C >= kMaxStride || a.x_stride < a.C || a.x_stride >= far)
        return GDN2_ERR_SHAPE;
    const int64_t es = elem(dtype);
    int64_t nx, ny, ns;
    if (!span(tokens, a.x_stride, a.C, es, &nx) || !span(tokens, a.C, a.C, es, &ny) || !mul_ok(a.N, a.C * 3 * es, &ns))
        return GDN2_ERR_SHAPE;
    // Threads of a launch, of four channels each: of a run of 16 tokens (shorter runs are for small
    // calls), and of a sequence's state.
    int64_t runs;
    if (!mul_ok(a.cu_seqlens ? 1 : a.N, (a.T + 15) / 16, &runs) || runs > INT64_MAX / 4 - a.N ||
        !mul_ok(runs + a.N, a.C / 4, &runs) || runs > UINT32_MAX - 1024)
        return GDN2_ERR_SHAPE;
    if (a.x && !aligned_to(a.x, es)) return GDN2_ERR_MISALIGNED;
    for (const void* p : {(const void*)a.taps, (const void*)a.bias, a.initial_state, (const void*)a.y, (const void*)a.final_state})
        if (p && !aligned_to(p, 16)) return GDN2_ERR_MISALIGNED;
    const Range ry = range_of(a.y, ny), rf = range_of(a.final_state, a.final_state ? ns : 0);
    const Range rc = range_of(a.cu_seqlens, a.cu_seqlens ? (a.N + 1) * 8 : 0);
    for (const Range& r : {range_of(a.x, nx), range_of(a.taps, a.C * 16), range_of(a.bias, a.bias ? a.C * 4 : 0), rc})
        if (overlap(ry, r) || overlap(rf, r)) return GDN2_ERR_ALIAS;
    const Range ri = range_of(a.initial_state, a.initial_state ? ns : 0);
    if (overlap(ry, rf) || overlap(ry, ri)) return GDN2_ERR_ALIAS;
    if (a.initial_state != a.final_state && overlap(ri, rf)) return GDN2_ERR_ALIAS;
    return GDN2_OK;
}

bool norm_sizes_ok(int64_t rows, int64_t width) { return rows >= 0 && rows <= INT_MAX && width >= 1 && width <= kMaxWidth; }

}  // namespace

extern "C" {

size_t gdn2_ssm_fwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv, gdn2_dtype_t dtype) {
    return ssm_workspace(false, B, T, H, dk, dv, dtype);
}

size_t gdn2_ssm_fwd_varlen_workspace_bytes(int64_t N, int64_t total_T, int64_t H, int64_t dk, int64_t dv,
                                           gdn2_dtype_t dtype) {
    return ssm_workspace(true, N, total_T, H, dk, dv, dtype);
}

gdn2_status_t gdn2_ssm_fwd(const void* x, const void* dt, const void* b, const void* c, const float* A, const float* D,
                           const float* dt_bias, const float* initial_state, void* y, float* final_state, int64_t B,
                           int64_t T, int64_t H, int64_t G, int64_t dk, int64_t dv, int64_t x_stride, int64_t dt_stride,
                           int64_t b_stride, int64_t c_stride, gdn2_dtype_t dtype, int softplus, void* workspace,
                           size_t workspace_bytes, void* stream) {
    int64_t tokens;
    if (B < 1 || T < 1 || !mul_ok(B, T, &tokens)) return GDN2_ERR_SHAPE;
    const gdn2::SsmArgs a{x, dt, b, c, A, D, dt_bias, initial_state, y, final_state, B, T, H, G, dk, dv, x_stride,
                          dt_stride, b_stride, c_stride, dtype == GDN2_DTYPE_BF16, softplus != 0, nullptr, stream, 0};
    return ssm_fwd(a, dtype, tokens, workspace, workspace_bytes);
}

gdn2_status_t gdn2_ssm_fwd_varlen(const void* x, const void* dt, const void* b, const void* c, const float* A,
                                  const float* D, const float* dt_bias, const float* initial_state, void* y,
                                  float* final_state, const int64_t* cu_seqlens, int64_t N, int64_t total_T, int64_t H,
                                  int64_t G, int64_t dk, int64_t dv, int64_t x_stride, int64_t dt_stride,
                                  int64_t b_stride, int64_t c_stride, gdn2_dtype_t dtype, int softplus, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    if (!cu_seqlens) return GDN2_ERR_NULL;
    if (!aligned_to(cu_seqlens, 8)) return GDN2_ERR_MISALIGNED;
    const gdn2::SsmArgs a{x, dt, b, c, A, D, dt_bias, initial_state, y, final_state, N, total_T, H, G, dk, dv, x_stride,
                          dt_stride, b_stride, c_stride, dtype == GDN2_DTYPE_BF16, softplus != 0, cu_seqlens, stream, 0};
    return ssm_fwd(a, dtype, total_T, workspace, workspace_bytes);
}

gdn2_status_t gdn2_ssm_step(const void* x, const void* dt, const void* b, const void* c, const float* A, const float* D,
                            const float* dt_bias, float* state, void* y, int64_t N, int64_t H, int64_t G, int64_t dk,
                            int64_t dv, int64_t x_stride, int64_t dt_stride, int64_t b_stride, int64_t c_stride,
                            gdn2_dtype_t dtype, int softplus, void* stream) {
    gdn2::SsmArgs a{x, dt, b, c, A, D, dt_bias, state, y, state, N, 1, H, G, dk, dv, x_stride, dt_stride, b_stride,
                    c_stride, dtype == GDN2_DTYPE_BF16, softplus != 0, nullptr, stream, 0};
    const gdn2_status_t st = check_ssm(a, dtype, N, true);
    if (st != GDN2_OK) return st;
    return gdn2::launch_ssm_step(a) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status_t gdn2_short_conv(const void* x, const float* taps, const float* bias, const void* initial_state, void* y,
                              void* final_state, int64_t B, int64_t T, int64_t C, int64_t x_stride, gdn2_dtype_t dtype,
                              void* stream) {
    int64_t tokens;
    if (B < 1 || T < 1 || !mul_ok(B, T, &tokens)) return GDN2_ERR_SHAPE;
    gdn2::ConvArgs a{x, taps, bias, initial_state, y, final_state, B, T, C, x_stride, dtype == GDN2_DTYPE_BF16,
                     nullptr, stream};
    const gdn2_status_t st = check_conv(a, dtype, tokens, false);
    if (st != GDN2_OK) return st;
    return gdn2::launch_short_conv(a) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status_t gdn2_short_conv_varlen(const void* x, const float* taps, const float* bias, const void* initial_state,
                                     void* y, void* final_state, const int64_t* cu_seqlens, int64_t N, int64_t total_T,
                                     int64_t C, int64_t x_stride, gdn2_dtype_t dtype, void* stream) {
    if (!cu_seqlens) return GDN2_ERR_NULL;
    if (!aligned_to(cu_seqlens, 8)) return GDN2_ERR_MISALIGNED;
    gdn2::ConvArgs a{x, taps, bias, initial_state, y, final_state, N, total_T, C, x_stride, dtype == GDN2_DTYPE_BF16,
                     cu_seqlens, stream};
    const gdn2_status_t st = check_conv(a, dtype, total_T, false);
    if (st != GDN2_OK) return st;
    if (total_T == 0 && !final_state) return GDN2_OK;
    return gdn2::launch_short_conv(a) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status_t gdn2_short_conv_step(const void* x, const float* taps, const float* bias, void* state, void* y, int64_t N,
                                   int64_t C, int64_t x_stride, gdn2_dtype_t dtype, void* stream) {
    gdn2::ConvArgs a{x, taps, bias, state, y, state, N, 1, C, x_stride, dtype == GDN2_DTYPE_BF16, nullptr, stream};
    const gdn2_status_t st = check_conv(a, dtype, N, true);
    if (st != GDN2_OK) return st;
    return gdn2::launch_short_conv_step(a) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status_t gdn2_layer_norm(const void* x, const float* gamma, const float* beta, void* y, float* mean, float* rstd,
                              int64_t rows, int64_t width, float eps, gdn2_dtype_t dtype, void* stream) {
    if (!known(dtype)) return GDN2_ERR_UNSUPPORTED;
    if (!norm_sizes_ok(rows, width) || !(eps >= 0.f) || eps > 1e30f) return GDN2_ERR_SHAPE;
    if (rows == 0) return GDN2_OK;
    if (!x || !gamma || !y || !mean != !rstd) return GDN2_ERR_NULL;
    for (const void* p : {x, (const void*)gamma, (const void*)beta, (const void*)y})
        if (p && !aligned_to(p, 16)) return GDN2_ERR_MISALIGNED;
    if (!aligned_to(mean, 4) || !aligned_to(rstd, 4)) return GDN2_ERR_MISALIGNED;
    const int64_t n = rows * width * elem(dtype), st = mean ? rows * 4 : 0;
    const Range outs[] = {range_of(y, n), range_of(mean, st), range_of(rstd, st)};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : {range_of(x, n), range_of(gamma, width * 4), range_of(beta, beta ? width * 4 : 0)})
            if (overlap(outs[i], r)) return GDN2_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return GDN2_ERR_ALIAS;
    }
    gdn2::NormArgs a{x, gamma, beta, y, mean, rstd, rows, width, dtype == GDN2_DTYPE_BF16, eps, stream};
    return gdn2::launch_layer_norm(a) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

size_t gdn2_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t width) {
    return norm_sizes_ok(rows, width) ? gdn2::norm_bwd_workspace_bytes(rows, width) : 0;
}

gdn2_status_t gdn2_layer_norm_bwd(const void* dy, const void* x, const float* gamma, const float* mean,
                                  const float* rstd, void* dx, float* dgamma, float* dbeta, void* workspace,
                                  size_t workspace_bytes, int64_t rows, int64_t width, gdn2_dtype_t dtype,
                                  void* stream) {
    if (!known(dtype)) return GDN2_ERR_UNSUPPORTED;
    if (!norm_sizes_ok(rows, width)) return GDN2_ERR_SHAPE;
    if (!gamma || !dgamma || (rows > 0 && (!dy || !x || !mean || !rstd || !dx))) return GDN2_ERR_NULL;
    for (const void* p : {dy, x, (const void*)gamma, (const void*)dx, (const void*)dgamma, (const void*)dbeta})
        if (p && !aligned_to(p, 16)) return GDN2_ERR_MISALIGNED;
    if (!aligned_to(mean, 4) || !aligned_to(rstd, 4)) return GDN2_ERR_MISALIGNED;
    const size_t need = gdn2_layer_norm_bwd_workspace_bytes(rows, width);
    if (need && (!workspace || workspace_bytes < need)) return GDN2_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return GDN2_ERR_MISALIGNED;
    const int64_t n = rows * width * elem(dtype);
    const Range outs[] = {range_of(dx, n), range_of(dgamma, width * 4), range_of(dbeta, dbeta ? width * 4 : 0),
                          range_of(workspace, (int64_t)need)};
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : {range_of(dy, n), range_of(x, n), range_of(gamma, width * 4), range_of(mean, rows * 4),
                               range_of(rstd, rows * 4)})
            if (overlap(outs[i], r)) return GDN2_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return GDN2_ERR_ALIAS;
    }
    gdn2::NormBwdArgs a{dy, x, gamma, mean, rstd, dx, dgamma, dbeta, static_cast<float*>(workspace), rows, width,
                        dtype == GDN2_DTYPE_BF16, stream};
    return gdn2::launch_layer_norm_bwd(a) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

}  // extern "C"
