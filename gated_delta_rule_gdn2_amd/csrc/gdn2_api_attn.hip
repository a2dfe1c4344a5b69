// gdn2_api_attn.hip -- the C ABI of the attention block (include/gdn2.h): attention, its gradients and
// its single-token step, rotary positions and the root-mean-square norm.  Argument validation and
// dispatch, on the host; nothing is enqueued before every check has passed.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>
#include <initializer_list>

#include "../../include/gdn2.h"
#include "gdn2_check.h"
#include "gdn2_launch.h"

namespace {

using gdn2::aligned_to;
using gdn2::mul_ok;
using gdn2::overlap;
using gdn2::Range;
using gdn2::range_of;

constexpr int64_t kMaxStride = int64_t(1) << 22;  // elements between tokens: 128 of them stay below 2^31 bytes
constexpr int64_t kMaxStepStride = int64_t(1) << 31;  // and between a step's, which are multiplied in 64 bits
constexpr int64_t kMaxStepGroups = int64_t(1) << 23;  // workgroups of a step that takes each sequence whole
constexpr int64_t kMaxWidth = 16384;
constexpr int64_t kMaxRotaryHead = 512;
// Tokens of a sequence, or of all packed ones: positions a few tiles behind the last stay 32-bit.
constexpr int64_t kMaxTokens = INT_MAX - 1024;

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

// compute units of the current device; without one (sizes asked for on a host) an MI355X's
int cus_or_default() {
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 256;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) return 256;
    return cus;
}

bool any_overlap(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range* a = outs.begin(); a != outs.end(); ++a) {
        for (const Range& b : ins)
            if (overlap(*a, b)) return true;
        for (const Range* b = outs.begin(); b != a; ++b)
            if (overlap(*a, *b)) return true;
    }
    return false;
}

// The bytes that attention's tensors take.
struct AttnBytes {
    int64_t tokens_q, tokens_k, q, k, v, o, lse, kv;  // o: of o, its gradient and dq; kv: of dk and of dv
};

// The checks that the forward and the backward pass share; the tensors' sizes.
gdn2_status_t check_attn(const gdn2::AttnArgs& a, gdn2_dtype_t dtype, AttnBytes* b) {
    if (!known(dtype)) return GDN2_ERR_UNSUPPORTED;
    if (a.N < 1 || a.T < 0 || a.S < 0 || a.H < 1 || a.G < 1 || a.d < 1 || a.window < 0) return GDN2_ERR_SHAPE;
    if (!gdn2::attn_supported(a.d)) return GDN2_ERR_UNSUPPORTED;
    if (a.N > INT_MAX || a.T > kMaxTokens || a.S > kMaxTokens || a.H >= kMaxStride || a.H % a.G) return GDN2_ERR_SHAPE;
    if (!(a.scale > 0.f) || a.scale > 1e30f) return GDN2_ERR_SHAPE;
    if (a.H * a.d >= kMaxStride) return GDN2_ERR_SHAPE;
    if (a.q_stride < a.H * a.d || a.k_stride < a.G * a.d || a.v_stride < a.G * a.d) return GDN2_ERR_SHAPE;
    if (a.q_stride >= kMaxStride || a.k_stride >= kMaxStride || a.v_stride >= kMaxStride) return GDN2_ERR_SHAPE;
    const int64_t es = elem(dtype);
    b->tokens_q = a.T;
    b->tokens_k = a.S;
    if (!a.cu_q && (!mul_ok(a.N, a.T, &b->tokens_q) || !mul_ok(a.N, a.S, &b->tokens_k))) return GDN2_ERR_SHAPE;
    if (!span(b->tokens_q, a.q_stride, a.H * a.d, es, &b->q) || !span(b->tokens_k, a.k_stride, a.G * a.d, es, &b->k) ||
        !span(b->tokens_k, a.v_stride, a.G * a.d, es, &b->v) || !span(b->tokens_q, a.H * a.d, a.H * a.d, 4, &b->o) ||
        !span(b->tokens_k, a.G * a.d, a.G * a.d, 4, &b->kv))
        return GDN2_ERR_SHAPE;
    b->o = b->o / 4 * es;
    b->kv = b->kv / 4 * es;
    b->lse = b->tokens_q * a.H * 4;
    if ((b->q && !a.q) || (b->k && (!a.k || !a.v))) return GDN2_ERR_NULL;
    if (!gdn2::attn_grid_ok(a)) return GDN2_ERR_SHAPE;
    if ((a.q_stride * es | a.k_stride * es | a.v_stride * es) & 15) return GDN2_ERR_MISALIGNED;
    for (const void* p : {a.q, a.k, a.v, (const void*)a.o, a.d_o, (const void*)a.dq, (const void*)a.dk, (const void*)a.dv})
        if (p && !aligned_to(p, 16)) return GDN2_ERR_MISALIGNED;
    if (!aligned_to(a.lse, 4)) return GDN2_ERR_MISALIGNED;
    return GDN2_OK;
}

gdn2_status_t attn_fwd(gdn2::AttnArgs a, gdn2_dtype_t dtype, void* workspace, size_t workspace_bytes) {
    AttnBytes b;
    const gdn2_status_t st = check_attn(a, dtype, &b);
    if (st != GDN2_OK) return st;
    if (b.o && !a.o) return GDN2_ERR_NULL;
    size_t need = 0;
    a.cus = cus_or_default();
    if (workspace || workspace_bytes) {
        need = b.tokens_q ? gdn2::attn_fwd_workspace_bytes(a) : 0;
        if (need == 0 || !workspace || workspace_bytes < need) return GDN2_ERR_WORKSPACE;
        if (!aligned_to(workspace, 16)) return GDN2_ERR_MISALIGNED;
    }
    const int64_t cu = a.cu_q ? (a.N + 1) * 8 : 0;
    if (any_overlap({range_of(a.o, b.o), range_of(a.lse, a.lse ? b.lse : 0), range_of(workspace, (int64_t)need)},
                    {range_of(a.q, b.q), range_of(a.k, b.k), range_of(a.v, b.v), range_of(a.cu_q, cu), range_of(a.cu_k, cu)}))
        return GDN2_ERR_ALIAS;
    if (b.tokens_q == 0) return GDN2_OK;
    return gdn2::launch_attn_fwd(a, workspace) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status_t attn_bwd(gdn2::AttnArgs a, gdn2_dtype_t dtype, void* workspace, size_t workspace_bytes) {
    AttnBytes b;
    const gdn2_status_t st = check_attn(a, dtype, &b);
    if (st != GDN2_OK) return st;
    if ((b.o && (!a.o || !a.d_o || !a.lse || !a.dq)) || (b.kv && (!a.dk || !a.dv))) return GDN2_ERR_NULL;
    a.cus = cus_or_default();
    const int64_t need = b.tokens_q ? (int64_t)gdn2::attn_bwd_workspace_bytes(a) : 0;
    if (need && (!workspace || workspace_bytes < (size_t)need)) return GDN2_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return GDN2_ERR_MISALIGNED;
    const int64_t cu = a.cu_q ? (a.N + 1) * 8 : 0;
    if (any_overlap({range_of(a.dq, b.o), range_of(a.dk, b.kv), range_of(a.dv, b.kv), range_of(workspace, need)},
                    {range_of(a.q, b.q), range_of(a.k, b.k), range_of(a.v, b.v), range_of(a.o, b.o), range_of(a.d_o, b.o),
                     range_of(a.lse, b.lse), range_of(a.cu_q, cu), range_of(a.cu_k, cu)}))
        return GDN2_ERR_ALIAS;
    if (b.tokens_q == 0 && b.tokens_k == 0) return GDN2_OK;
    return gdn2::launch_attn_bwd(a, workspace) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

size_t attn_workspace(size_t (*bytes)(const gdn2::AttnArgs&), bool packed, int64_t N, int64_t T, int64_t S, int64_t H, int64_t G,
                      int64_t d, int64_t window, gdn2_dtype_t dtype) {
    static const int64_t cu[2] = {0, 0};  // never read: says that sequences are packed
    gdn2::AttnArgs a{};
    a.N = N, a.T = T, a.S = S, a.H = H, a.G = G, a.d = d, a.window = window, a.scale = 1.f;
    a.dtype_bf16 = dtype == GDN2_DTYPE_BF16;
    if (H > 0 && G > 0 && d > 0 && H < kMaxStride && d < kMaxStride) a.q_stride = H * d, a.k_stride = a.v_stride = G * d;
    if (packed) a.cu_q = a.cu_k = cu;
    a.q = a.k = a.v = reinterpret_cast<const void*>(uintptr_t(16));  // never read
    AttnBytes b;
    if (check_attn(a, dtype, &b) != GDN2_OK || b.tokens_q == 0) return 0;
    a.cus = cus_or_default();
    return bytes(a);
}

// Tokens of `width` bytes each, `stride` bytes apart: whether two such tensors share a byte.  Parts of
// one wider tensor have the same stride and lie between each other's tokens.
struct Strided {
    const void* p;
    int64_t tokens, stride, width;
    Range range() const { return range_of(p, tokens > 0 ? (tokens - 1) * stride + width : 0); }
};
bool overlap(const Strided& a, const Strided& b) {
    if (!overlap(a.range(), b.range())) return false;
    if (a.stride != b.stride) return true;
    const int64_t apart = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % a.stride;
    const int64_t behind = apart < 0 ? apart + a.stride : apart;  // of b's token, behind the start of a token of a
    return behind < a.width || a.stride - behind < b.width;
}

gdn2_status_t attn_step(gdn2::AttnStepArgs a, gdn2_dtype_t dtype, void* workspace, size_t workspace_bytes) {
    if (!known(dtype)) return GDN2_ERR_UNSUPPORTED;
    if (a.N < 1 || a.H < 1 || a.G < 1 || a.d < 1 || a.C < 1 || a.window < 0) return GDN2_ERR_SHAPE;
    if (!gdn2::attn_supported(a.d)) return GDN2_ERR_UNSUPPORTED;
    if (!a.q || !a.k || !a.v || !a.k_cache || !a.v_cache || !a.positions || !a.o) return GDN2_ERR_NULL;
    if (a.N > INT_MAX || a.C > kMaxTokens || a.H >= kMaxStride || a.H % a.G || a.H * a.d >= kMaxStride) return GDN2_ERR_SHAPE;
    if (!(a.scale > 0.f) || a.scale > 1e30f) return GDN2_ERR_SHAPE;
    if (a.q_stride < a.H * a.d || a.k_stride < a.G * a.d || a.v_stride < a.G * a.d) return GDN2_ERR_SHAPE;
    if (a.q_stride >= kMaxStepStride || a.k_stride >= kMaxStepStride || a.v_stride >= kMaxStepStride) return GDN2_ERR_SHAPE;
    if (a.N * a.G * ((a.H / a.G + 31) / 32) >= kMaxStepGroups) return GDN2_ERR_SHAPE;
    const int64_t es = elem(dtype);
    int64_t nq, nk, nv, no, nc;
    if (!span(a.N, a.q_stride, a.H * a.d, es, &nq) || !span(a.N, a.k_stride, a.G * a.d, es, &nk) ||
        !span(a.N, a.v_stride, a.G * a.d, es, &nv) || !span(a.N, a.H * a.d, a.H * a.d, es, &no) || !mul_ok(a.N, a.C, &nc) ||
        !mul_ok(nc, a.G * a.d * es, &nc))
        return GDN2_ERR_SHAPE;
    if ((a.q_stride * es | a.k_stride * es | a.v_stride * es) & 15) return GDN2_ERR_MISALIGNED;
    for (const void* p : {a.q, a.k, a.v, (const void*)a.k_cache, (const void*)a.v_cache, (const void*)a.o})
        if (!aligned_to(p, 16)) return GDN2_ERR_MISALIGNED;
    if (!aligned_to(a.positions, 8)) return GDN2_ERR_MISALIGNED;
    size_t need = 0;
    if (workspace || workspace_bytes) {
        a.cus = cus_or_default();
        need = gdn2::attn_step_workspace_bytes(a);
        if (need == 0 || !workspace || workspace_bytes < need) return GDN2_ERR_WORKSPACE;
        if (!aligned_to(workspace, 16)) return GDN2_ERR_MISALIGNED;
    }
    if (any_overlap({range_of(a.o, no), range_of(a.k_cache, nc), range_of(a.v_cache, nc), range_of(workspace, (int64_t)need)},
                    {range_of(a.q, nq), range_of(a.k, nk), range_of(a.v, nv), range_of(a.positions, a.N * 8)}))
        return GDN2_ERR_ALIAS;
    return gdn2::launch_attn_step(a, workspace) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

bool rms_sizes_ok(int64_t rows, int64_t width) { return rows >= 0 && rows <= INT_MAX && width >= 1 && width <= kMaxWidth; }

gdn2_status_t rms_norm(const gdn2::RmsArgs& a, gdn2_dtype_t dtype, gdn2_dtype_t residual_dtype, int64_t out_bytes) {
    if (!known(dtype) || (a.residual && residual_dtype != dtype && residual_dtype != GDN2_DTYPE_F32)) return GDN2_ERR_UNSUPPORTED;
    if (!rms_sizes_ok(a.rows, a.width) || !(a.eps >= 0.f) || a.eps > 1e30f) return GDN2_ERR_SHAPE;
    if (a.rows == 0) return GDN2_OK;
    if (!a.x || !a.gamma || !a.y || !a.residual != !a.h) return GDN2_ERR_NULL;
    for (const void* p : {a.x, a.residual, (const void*)a.gamma, (const void*)a.y, (const void*)a.h})
        if (p && !aligned_to(p, 16)) return GDN2_ERR_MISALIGNED;
    if (!aligned_to(a.scale, 4) || !aligned_to(a.rstd, 4)) return GDN2_ERR_MISALIGNED;
    const int64_t n = a.rows * a.width, nr = a.residual ? n * elem(residual_dtype) : 0;
    const Range x = range_of(a.x, n * elem(dtype)), r = range_of(a.residual, nr), g = range_of(a.gamma, a.width * 4);
    const Range h = range_of(a.h, nr), y = range_of(a.y, n * out_bytes);
    const Range s = range_of(a.scale, a.scale ? a.rows * 4 : 0), t = range_of(a.rstd, a.rstd ? a.rows * 4 : 0);
    // the sum may take the residual's place
    if (any_overlap({y, s, t}, {x, r, g, h}) || overlap(h, x) || overlap(h, g) || (a.h != a.residual && overlap(h, r)))
        return GDN2_ERR_ALIAS;
    return gdn2::launch_rms_norm(a) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

}  // namespace

extern "C" {

size_t gdn2_attn_bwd_workspace_bytes(int64_t B, int64_t T, int64_t S, int64_t H, int64_t G, int64_t d, int64_t window,
                                     gdn2_dtype_t dtype) {
    return attn_workspace(gdn2::attn_bwd_workspace_bytes, false, B, T, S, H, G, d, window, dtype);
}

size_t gdn2_attn_bwd_varlen_workspace_bytes(int64_t N, int64_t total_T, int64_t total_S, int64_t H, int64_t G, int64_t d,
                                            int64_t window, gdn2_dtype_t dtype) {
    return attn_workspace(gdn2::attn_bwd_workspace_bytes, true, N, total_T, total_S, H, G, d, window, dtype);
}

gdn2_status_t gdn2_attn_bwd(const void* d_o, const void* q, const void* k, const void* v, const void* o, const float* lse,
                            void* dq, void* dk, void* dv, int64_t B, int64_t T, int64_t S, int64_t H, int64_t G, int64_t d,
                            int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t window, float scale,
                            gdn2_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const gdn2::AttnArgs a{q, k, v, const_cast<void*>(o), const_cast<float*>(lse), B, T, S, H, G, d, q_stride, k_stride,
                           v_stride, window, scale, dtype == GDN2_DTYPE_BF16, nullptr, nullptr, stream, 0, d_o, dq, dk, dv};
    return attn_bwd(a, dtype, workspace, workspace_bytes);
}

gdn2_status_t gdn2_attn_bwd_varlen(const void* d_o, const void* q, const void* k, const void* v, const void* o,
                                   const float* lse, void* dq, void* dk, void* dv, const int64_t* cu_seqlens,
                                   const int64_t* cu_seqlens_k, int64_t N, int64_t total_T, int64_t total_S, int64_t H,
                                   int64_t G, int64_t d, int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t window,
                                   float scale, gdn2_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (!cu_seqlens || !cu_seqlens_k) return GDN2_ERR_NULL;
    if (!aligned_to(cu_seqlens, 8) || !aligned_to(cu_seqlens_k, 8)) return GDN2_ERR_MISALIGNED;
    const gdn2::AttnArgs a{q, k, v, const_cast<void*>(o), const_cast<float*>(lse), N, total_T, total_S, H, G, d, q_stride,
                           k_stride, v_stride, window, scale, dtype == GDN2_DTYPE_BF16, cu_seqlens, cu_seqlens_k, stream, 0,
                           d_o, dq, dk, dv};
    return attn_bwd(a, dtype, workspace, workspace_bytes);
}

gdn2_status_t gdn2_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t T, int64_t S,
                            int64_t H, int64_t G, int64_t d, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                            int64_t window, float scale, gdn2_dtype_t dtype, void* workspace, size_t workspace_bytes,
                            void* stream) {
    const gdn2::AttnArgs a{q, k, v, o, lse, B, T, S, H, G, d, q_stride, k_stride, v_stride, window, scale,
                           dtype == GDN2_DTYPE_BF16, nullptr, nullptr, stream, 0};
    return attn_fwd(a, dtype, workspace, workspace_bytes);
}

gdn2_status_t gdn2_attn_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse, const int64_t* cu_seqlens,
                                   const int64_t* cu_seqlens_k, int64_t N, int64_t total_T, int64_t total_S, int64_t H,
                                   int64_t G, int64_t d, int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t window,
                                   float scale, gdn2_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (!cu_seqlens || !cu_seqlens_k) return GDN2_ERR_NULL;
    if (!aligned_to(cu_seqlens, 8) || !aligned_to(cu_seqlens_k, 8)) return GDN2_ERR_MISALIGNED;
    const gdn2::AttnArgs a{q, k, v, o, lse, N, total_T, total_S, H, G, d, q_stride, k_stride, v_stride, window, scale,
                           dtype == GDN2_DTYPE_BF16, cu_seqlens, cu_seqlens_k, stream, 0};
    return attn_fwd(a, dtype, workspace, workspace_bytes);
}

size_t gdn2_attn_fwd_workspace_bytes(int64_t B, int64_t T, int64_t S, int64_t H, int64_t G, int64_t d, int64_t window,
                                     gdn2_dtype_t dtype) {
    return attn_workspace(gdn2::attn_fwd_workspace_bytes, false, B, T, S, H, G, d, window, dtype);
}

size_t gdn2_attn_fwd_varlen_workspace_bytes(int64_t N, int64_t total_T, int64_t total_S, int64_t H, int64_t G, int64_t d,
                                            int64_t window, gdn2_dtype_t dtype) {
    return attn_workspace(gdn2::attn_fwd_workspace_bytes, true, N, total_T, total_S, H, G, d, window, dtype);
}

size_t gdn2_attn_step_workspace_bytes(int64_t N, int64_t H, int64_t G, int64_t d, int64_t C, int64_t window, gdn2_dtype_t dtype) {
    if (!known(dtype) || N < 1 || H < 1 || G < 1 || C < 1 || window < 0 || !gdn2::attn_supported(d)) return 0;
    if (N > INT_MAX || C > kMaxTokens || H >= kMaxStride || H % G || N * G * ((H / G + 31) / 32) >= kMaxStepGroups) return 0;
    gdn2::AttnStepArgs a{};
    a.N = N, a.H = H, a.G = G, a.d = d, a.C = C, a.window = window, a.dtype_bf16 = dtype == GDN2_DTYPE_BF16;
    a.cus = cus_or_default();
    return gdn2::attn_step_workspace_bytes(a);
}

gdn2_status_t gdn2_attn_step(const void* q, const void* k, const void* v, void* k_cache, void* v_cache, const int64_t* positions,
                             void* o, int64_t N, int64_t H, int64_t G, int64_t d, int64_t C, int64_t q_stride, int64_t k_stride,
                             int64_t v_stride, int64_t window, float scale, gdn2_dtype_t dtype, void* workspace,
                             size_t workspace_bytes, void* stream) {
    const gdn2::AttnStepArgs a{q, k, v, k_cache, v_cache, positions, o, N, H, G, d, C, q_stride, k_stride, v_stride, window, scale,
                               dtype == GDN2_DTYPE_BF16, stream, 0};
    return attn_step(a, dtype, workspace, workspace_bytes);
}

gdn2_status_t gdn2_rotary(const void* q, const void* k, const float* freq, const int64_t* positions, void* q_out, void* k_out,
                          int64_t tokens, int64_t T, int64_t H, int64_t G, int64_t d, int64_t rot, int64_t q_stride,
                          int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride, int interleaved, int inverse, float scale,
                          gdn2_dtype_t dtype, void* stream) {
    if (!known(dtype)) return GDN2_ERR_UNSUPPORTED;
    if (tokens < 0 || tokens > kMaxTokens || T < 1 || H < 1 || G < 0 || d < 2 || d > kMaxRotaryHead) return GDN2_ERR_SHAPE;
    if (rot < 2 || rot % 2 || rot > d || H >= kMaxStride || G >= kMaxStride || (H + G) * d >= kMaxStride) return GDN2_ERR_SHAPE;
    if (!(scale > 0.f) || scale > 1e30f) return GDN2_ERR_SHAPE;
    if (G == 0) {
        k = nullptr;
        k_out = nullptr;
        k_stride = k_out_stride = 0;
    }
    if (q_stride < H * d || q_out_stride < H * d || k_stride < G * d || k_out_stride < G * d) return GDN2_ERR_SHAPE;
    for (int64_t s : {q_stride, k_stride, q_out_stride, k_out_stride})
        if (s >= kMaxStepStride) return GDN2_ERR_SHAPE;
    if (tokens == 0) return GDN2_OK;
    if (!q || !q_out || !freq || (G > 0 && (!k || !k_out))) return GDN2_ERR_NULL;
    const int64_t es = elem(dtype);
    for (const void* p : {q, (const void*)q_out, k, (const void*)k_out})
        if (!aligned_to(p, es)) return GDN2_ERR_MISALIGNED;
    if (!aligned_to(freq, 4) || !aligned_to(positions, 8)) return GDN2_ERR_MISALIGNED;
    const Strided qi{q, tokens, q_stride * es, H * d * es}, qo{q_out, tokens, q_out_stride * es, H * d * es};
    const Strided ki{k, G ? tokens : 0, k_stride * es, G * d * es}, ko{k_out, G ? tokens : 0, k_out_stride * es, G * d * es};
    const Range f = range_of(freq, rot / 2 * 4), p = range_of(positions, positions ? tokens * 8 : 0);
    for (const Strided* s : {&qo, &ko})
        if (overlap(s->range(), f) || overlap(s->range(), p)) return GDN2_ERR_ALIAS;
    if (!(q == q_out && q_stride == q_out_stride) && overlap(qi, qo)) return GDN2_ERR_ALIAS;
    if (G && !(k == k_out && k_stride == k_out_stride) && overlap(ki, ko)) return GDN2_ERR_ALIAS;
    if (G && (overlap(qo, ki) || overlap(ko, qi) || overlap(qo, ko))) return GDN2_ERR_ALIAS;
    const gdn2::RotaryArgs a{q, k, freq, positions, q_out, k_out, tokens, T, H, G, d, rot / 2, q_stride, k_stride, q_out_stride,
                             k_out_stride, scale, dtype == GDN2_DTYPE_BF16, interleaved != 0, inverse != 0, stream};
    if (!gdn2::rotary_grid_ok(a)) return GDN2_ERR_SHAPE;
    return gdn2::launch_rotary(a) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status_t gdn2_rms_norm(const void* x, const void* residual, const float* gamma, void* y, void* h, float* rstd, int64_t rows,
                            int64_t width, float eps, gdn2_dtype_t dtype, gdn2_dtype_t residual_dtype, void* stream) {
    const gdn2::RmsArgs a{x, residual, gamma, y, nullptr, h, rstd, rows, width, dtype == GDN2_DTYPE_BF16,
                          residual ? residual_dtype == GDN2_DTYPE_BF16 : dtype == GDN2_DTYPE_BF16, eps, stream};
    return rms_norm(a, dtype, residual_dtype, elem(dtype));
}

gdn2_status_t gdn2_rms_norm_fp8(const void* x, const void* residual, const float* gamma, void* y, float* scales, void* h,
                                float* rstd, int64_t rows, int64_t width, float eps, gdn2_dtype_t dtype,
                                gdn2_dtype_t residual_dtype, void* stream) {
    if (rows > 0 && !scales) return GDN2_ERR_NULL;
    const gdn2::RmsArgs a{x, residual, gamma, y, scales, h, rstd, rows, width, dtype == GDN2_DTYPE_BF16,
                          residual ? residual_dtype == GDN2_DTYPE_BF16 : dtype == GDN2_DTYPE_BF16, eps, stream};
    return rms_norm(a, dtype, residual_dtype, 1);
}

size_t gdn2_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t width) {
    return rms_sizes_ok(rows, width) ? gdn2::rms_bwd_workspace_bytes(rows, width) : 0;
}

gdn2_status_t gdn2_rms_norm_bwd(const void* dy, const void* h, const float* gamma, const float* rstd, const void* dh, void* dx,
                                float* dgamma, void* workspace, size_t workspace_bytes, int64_t rows, int64_t width,
                                gdn2_dtype_t dtype, gdn2_dtype_t residual_dtype, void* stream) {
    if (!known(dtype) || (residual_dtype != dtype && residual_dtype != GDN2_DTYPE_F32)) return GDN2_ERR_UNSUPPORTED;
    if (!rms_sizes_ok(rows, width)) return GDN2_ERR_SHAPE;
    if (!gamma || !dgamma || (rows > 0 && (!dy || !h || !rstd || !dx))) return GDN2_ERR_NULL;
    for (const void* p : {dy, h, (const void*)gamma, dh, (const void*)dx, (const void*)dgamma})
        if (p && !aligned_to(p, 16)) return GDN2_ERR_MISALIGNED;
    if (!aligned_to(rstd, 4)) return GDN2_ERR_MISALIGNED;
    const size_t need = gdn2_rms_norm_bwd_workspace_bytes(rows, width);
    if (need && (!workspace || workspace_bytes < need)) return GDN2_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return GDN2_ERR_MISALIGNED;
    const int64_t n = rows * width, nh = n * elem(residual_dtype);
    const Range x = range_of(dx, nh), d = range_of(dh, dh ? nh : 0);
    // dx may take dh's place
    if (any_overlap({x, range_of(dgamma, width * 4), range_of(workspace, (int64_t)need)},
                    {range_of(dy, n * elem(dtype)), range_of(h, nh), range_of(gamma, width * 4), range_of(rstd, rows * 4)}) ||
        overlap(range_of(dgamma, width * 4), d) || overlap(range_of(workspace, (int64_t)need), d) || (dx != dh && overlap(x, d)))
        return GDN2_ERR_ALIAS;
    const gdn2::RmsBwdArgs a{dy, h, gamma, rstd, dh, dx, dgamma, static_cast<float*>(workspace), rows, width,
                             dtype == GDN2_DTYPE_BF16, residual_dtype == GDN2_DTYPE_BF16, stream};
    return gdn2::launch_rms_norm_bwd(a) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

}  // extern "C"
