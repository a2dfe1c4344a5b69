// gdn2_attn_bwd.hip -- gradients of causal attention, which forms the probabilities again.
//
//   P_ij = e^(scale q_i . k_j - lse_i) for the keys j that query i sees (0 for the others),
//   delta_i = d_o_i . o_i,  dP_ij = d_o_i . v_j,  dS_ij = P_ij (dP_ij - delta_i),
//   dv_j = sum_i P_ij d_o_i,  dk_j = scale sum_i dS_ij q_i,  dq_i = scale sum_j dS_ij k_j,
// the sums over i also over the query heads that share a key head.
//
// Three kernels: delta and lse in base 2 (`stats`), then one workgroup a block of keys for dk and dv,
// then one a block of queries for dq.  Every sum is formed by one wave in a fixed order: equal calls
// give equal bits, at the price of S and dP twice (7 products instead of 5; partial sums of dq for
// each block of keys would move more bytes than that takes).  Sums are fp32; with bf16 inputs P and dS
// are rounded to bf16 once, as the matrix unit's operands, and gradients on the store.
#include "gdn2_attn.h"

namespace gdn2 {
namespace attn {

struct BwdParams {
    const char* q;
    const char* k;
    const char* v;
    const char* o;
    const char* d_o;
    const float* lse;
    void* dq;
    void* dk;
    void* dv;
    float2* stats;   // [heads][tokens]: lse in base 2, delta
    int64_t tokens;  // queries in all
    Shape p;
};

// ---- lse in base 2 and delta ------------------------------------------------------------------

constexpr int kStatTokens = 64, kStatHeads = 4;

// 64 tokens of 4 heads a workgroup: rows are read as they lie, 16 bytes a lane, and go out with a
// head's tokens side by side
template <typename T, int D>
__global__ __launch_bounds__(256) void stats_kernel(BwdParams a) {
    constexpr int V = 16 / (int)sizeof(T), LPR = D / V, RPP = 256 / LPR;  // lanes a row, rows at a time
    __shared__ float delta[kStatHeads][kStatTokens];
    const int64_t t0 = (int64_t)blockIdx.x * kStatTokens;
    const int h0 = blockIdx.y * kStatHeads, heads = a.p.heads, lane = threadIdx.x % LPR;
    for (int r = threadIdx.x / LPR; r < kStatTokens * kStatHeads; r += RPP) {
        const int t = r / kStatHeads, h = r % kStatHeads;
        float sum = 0.f;
        if (t0 + t < a.tokens && h0 + h < heads) {
            const int64_t at = ((t0 + t) * heads + h0 + h) * D + lane * V;
            const Vec<T, V> x = load_vec<T, V>(reinterpret_cast<const T*>(a.o) + at);
            const Vec<T, V> y = load_vec<T, V>(reinterpret_cast<const T*>(a.d_o) + at);
#pragma unroll
            for (int e = 0; e < V; ++e) sum += to_f32(x.v[e]) * to_f32(y.v[e]);
        }
#pragma unroll
        for (int s = LPR / 2; s >= 1; s /= 2) sum += __shfl_xor(sum, s);
        if (lane == 0) delta[h][t] = sum;
    }
    __syncthreads();
    const int t = threadIdx.x % kStatTokens, h = threadIdx.x / kStatTokens;
    if (t0 + t < a.tokens && h0 + h < heads)
        a.stats[(int64_t)(h0 + h) * a.tokens + t0 + t] =
            float2{a.lse[(t0 + t) * heads + h0 + h] * kLog2e, delta[h][t]};
}

// ---- dk and dv --------------------------------------------------------------------------------

constexpr int kQueries = 32;  // queries in a tile

template <typename T, int D, int NW>
__global__ __launch_bounds__(NW * 64, D * sizeof(T) > 128 ? 1 : 2) void dkv_kernel(BwdParams a) {
    typedef Tile<T, D> L;
    constexpr int KS = D / 16, DT = D / 32, BN = NW * 32, BQ = kQueries, BYTES = BQ * L::kRow, STAGE = 2 * BYTES + 1024;
    __shared__ __attribute__((aligned(1024))) char lds[2 * STAGE];
    __shared__ int special;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Shape& p = a.p;
    Work w;
    if (!find_work(p, BN, 1, false, true, lane, &w)) return;
    w = uniform(w);
    const int kv = w.head, share = p.heads / p.groups, lq = w.s.lq, lk = w.s.lk;
    const int first = w.block * BN, mine = first + wave * 32, rows = min(32, lk - mine);
    const int64_t off = (int64_t)lk - lq;  // where query 0 stands

    // the wave's keys and values; a lane's own is column l % 32
    Op<T> k[KS], v[KS];
    {
        const auto rk = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(a.k + (w.s.k0 + mine) * p.k_stride + (int64_t)kv * L::kRow), 0,
                                                          span(rows, p.k_stride, L::kRow), 0x00020000);
        const auto rv = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(a.v + (w.s.k0 + mine) * p.v_stride + (int64_t)kv * L::kRow), 0,
                                                          span(rows, p.v_stride, L::kRow), 0x00020000);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            k[ks] = global_op<T>(rk, (lane & 31) * p.k_stride, ks, g);
            v[ks] = global_op<T>(rv, (lane & 31) * p.v_stride, ks, g);
        }
    }
    f32x16 dk[DT], dv[DT];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) dk[dt] = dv[dt] = zero16();

    // tiles of the queries that see some key of the block; the heads one after the other
    const int64_t from = first - off, to = min((int64_t)first + BN, (int64_t)lk) - 1 - off + p.window;  // [from, to)
    const int t0 = from > 0 ? (int)(min(from, (int64_t)lq) / BQ) : 0;
    const int t1 = to > 0 ? (int)((min(to, (int64_t)lq) + BQ - 1) / BQ) : 0;
    const uint32_t o_stride = (uint32_t)p.heads * L::kRow;
    const Lds base = lds_of(lds), row_base = L::row_base(lane), col_base = L::col_base(lane);
    auto stage = [&](int h, int t, int buf) {
        const int head = kv * share + h, left = min(BQ, lq - t * BQ);
        const int64_t token = w.s.q0 + (int64_t)t * BQ;
        const Lds at = base + buf * STAGE;
        L::template stage<BQ, NW>(at, a.q + token * p.q_stride + (int64_t)head * L::kRow, span(left, p.q_stride, L::kRow), p.q_stride, wave, lane);
        L::template stage<BQ, NW>(at + BYTES, a.d_o + token * o_stride + (int64_t)head * L::kRow, span(left, o_stride, L::kRow), o_stride, wave, lane);
        if (wave == 0) load_words_to_lds(at + 2 * BYTES, rsrc_words(a.stats + (int64_t)head * a.tokens + token, left * 8), lane * 4);
    };
    if (tid == 0) special = -1;
    const int count = t1 > t0 ? share * (t1 - t0) : 0;
    int h = 0, t = t0;
    if (count > 0) stage(h, t, 0);
    for (int n = 0; n < count; ++n) {
        tile_barrier();
        int next_h = h, next_t = t + 1;
        if (next_t == t1) {
            next_t = t0;
            ++next_h;
        }
        if (n + 1 < count) stage(next_h, next_t, (n + 1) & 1);
        const Lds tq = base + (n & 1) * STAGE, tdo = tq + BYTES, ts = tdo + BYTES;
        const int64_t place = off + (int64_t)t * BQ;  // of the tile's first query
        const bool idle = rows <= 0 || place + BQ - 1 < mine || place > (int64_t)mine + 30 + p.window;
        // some query of the tile does not see some key of the block, or is none
        const bool cut = place < (int64_t)first + BN - 1 || place + BQ - 1 >= (int64_t)first + p.window || (t + 1) * (int64_t)BQ > lq;
        bool found = false;
        if (cut) {
            if (any_special<T, 2 * BYTES, NW * 64>(tq, tid)) special = n;
            __syncthreads();
            found = special == n;
        }
        // the queries that see the lane's key
        Seen seen{0, BQ};
        if (cut) {
            const int64_t lo = (int64_t)mine + (lane & 31) - place, hi = min(lo + p.window - 1, (int64_t)lq - 1 - (int64_t)t * BQ);
            seen = seen_between((int)max(lo, (int64_t)-1), (int)max((int64_t)-2, min(hi, (int64_t)BQ)));
        }
        Op<T> pr[BQ / 16], ds[BQ / 16];
        if (!idle) {
            const Lds rq = opaque(row_base + tq), ro = opaque(row_base + tdo);
            f32x16 s = zero16(), dp = zero16();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) mma(s, L::row_op(rq, 0, ks), k[ks]);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) mma(dp, L::row_op(ro, 0, ks), v[ks]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const f32x4 x = lds_get<f32x4>(ts + (8 * c + 4 * g) * 8), y = lds_get<f32x4>(ts + (8 * c + 4 * g) * 8 + 16);
                const float lse[4] = {x[0], x[2], y[0], y[2]}, delta[4] = {x[1], x[3], y[1], y[3]};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 4 * c + e;
                    s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], p.scale_log2, -lse[e]));
                    dp[i] = s[i] * (dp[i] - delta[e]);
                }
            }
            if (cut) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const bool yes = seen(acc_row(i, g));
                    s[i] = yes ? s[i] : 0.f;
                    dp[i] = yes ? dp[i] : 0.f;
                }
            }
#pragma unroll
            for (int c = 0; c < BQ / 16; ++c) {
                pr[c] = op_of<T>(s, c);
                ds[c] = op_of<T>(dp, c);
            }
        }
        if (found) {
            // a query that is not finite has made its dS a NaN where it sees the key; its d_o adds to dv
            if (!idle) {
                f32x16 add[DT];
                special_sums<T, D, BQ>(add, col_base + tdo, seen, g, false);
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) dv[dt] += add[dt];
            }
            __syncthreads();
            clear_special<T, 2 * BYTES, NW * 64>(tq, tid);
            __syncthreads();
        }
        if (!idle) {
            const Lds cq = opaque(col_base + tq), co = opaque(col_base + tdo);
#pragma unroll
            for (int c = 0; c < BQ / 16; ++c)
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) {
                    mma(dv[dt], L::col_op(co, 16 * c, dt), pr[c]);
                    mma(dk[dt], L::col_op(cq, 16 * c, dt), ds[c]);
                }
        }
        h = next_h;
        t = next_t;
    }
    if ((lane & 31) >= rows) return;
    const int64_t at = ((w.s.k0 + mine + (lane & 31)) * p.groups + kv) * D;
    store_column<T, D>(reinterpret_cast<T*>(a.dk) + at, dk, p.scale, g);
    store_column<T, D>(reinterpret_cast<T*>(a.dv) + at, dv, 1.f, g);
}

// ---- dq ---------------------------------------------------------------------------------------

template <typename T> constexpr int kKeys = sizeof(T) == 2 ? 64 : 32;  // keys in a tile

template <typename T, int D, int NW>
__global__ __launch_bounds__(NW * 64, D * sizeof(T) > 256 ? 1 : 2) void dq_kernel(BwdParams a) {
    typedef Tile<T, D> L;
    constexpr int BK = kKeys<T>, KS = D / 16, DT = D / 32, BM = NW * 32, BYTES = BK * L::kRow;
    __shared__ __attribute__((aligned(1024))) char lds[2 * 2 * BYTES];
    __shared__ int special;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Shape& p = a.p;
    Work w;
    if (!find_work(p, BM, p.heads / p.groups, true, false, lane, &w)) return;
    w = uniform(w);
    const int head = w.head, kv = head / (p.heads / p.groups), lq = w.s.lq, lk = w.s.lk;
    const char* kp = a.k + w.s.k0 * p.k_stride + (int64_t)kv * L::kRow;
    const char* vp = a.v + w.s.k0 * p.v_stride + (int64_t)kv * L::kRow;
    const int first = w.block * BM, off = lk - lq;
    const int64_t low = (int64_t)off + first, high = off + (int64_t)min(first + BM, lq) - 1;
    const int64_t from = low - p.window + 1;
    const int t0 = from > 0 ? (int)(from / BK) : 0, t1 = high >= 0 ? (int)(high / BK) + 1 : 0;
    const int mine = first + wave * 32, rows = min(32, lq - mine);
    const int64_t pos0 = (int64_t)off + mine;
    const int pos = (int)(pos0 + (lane & 31));
    const uint32_t o_stride = (uint32_t)p.heads * L::kRow;

    Op<T> q[KS], d_o[KS];
    float lse, delta;
    {
        const auto rq = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(a.q + (w.s.q0 + mine) * p.q_stride + (int64_t)head * L::kRow), 0,
                                                          span(rows, p.q_stride, L::kRow), 0x00020000);
        const auto ro = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(a.d_o + (w.s.q0 + mine) * o_stride + (int64_t)head * L::kRow), 0,
                                                          span(rows, o_stride, L::kRow), 0x00020000);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            q[ks] = global_op<T>(rq, (lane & 31) * p.q_stride, ks, g);
            d_o[ks] = global_op<T>(ro, (lane & 31) * o_stride, ks, g);
        }
        const bool live = (lane & 31) < rows;
        const float2 s = live ? a.stats[(int64_t)head * a.tokens + w.s.q0 + mine + (lane & 31)] : float2{0.f, 0.f};
        lse = s.x;
        delta = s.y;
    }
    f32x16 dq[DT];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) dq[dt] = zero16();
    const Lds base = lds_of(lds), row_base = L::row_base(lane), col_base = L::col_base(lane);
    auto stage = [&](int t) {
        const Lds at = base + (t & 1) * 2 * BYTES;
        const int left = min(BK, lk - t * BK);
        L::template stage<BK, NW>(at, kp + (int64_t)t * BK * p.k_stride, span(left, p.k_stride, L::kRow), p.k_stride, wave, lane);
        L::template stage<BK, NW>(at + BYTES, vp + (int64_t)t * BK * p.v_stride, span(left, p.v_stride, L::kRow), p.v_stride, wave, lane);
    };
    if (tid == 0) special = -1;
    if (t0 < t1) stage(t0);
    for (int t = t0; t < t1; ++t) {
        tile_barrier();
        if (t + 1 < t1) stage(t + 1);
        const Lds tk = base + (t & 1) * 2 * BYTES, tv = tk + BYTES;
        const int key0 = t * BK;
        const bool idle = rows <= 0 || key0 > pos0 + rows - 1 || key0 + BK - 1 <= pos0 - p.window;
        const Seen seen = seen_between(pos - key0 - p.window + 1, pos - key0);
        const bool cut = key0 + BK - 1 > low || key0 <= low + BM - 1 - p.window;
        bool found = false;
        if (cut) {
            if (any_special<T, BYTES, NW * 64>(tk, tid)) special = t;
            __syncthreads();
            found = special == t;
        }
        Op<T> ds[BK / 16];
        if (!idle) {
            const Lds rk = opaque(row_base + tk), rv = opaque(row_base + tv);
#pragma unroll
            for (int h = 0; h < BK / 32; ++h) {
                f32x16 s = zero16(), dp = zero16();
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) mma(s, L::row_op(rk, 32 * h, ks), q[ks]);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) mma(dp, L::row_op(rv, 32 * h, ks), d_o[ks]);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], p.scale_log2, -lse));
                    dp[i] = s[i] * (dp[i] - delta);
                }
                if (cut) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) dp[i] = seen(32 * h + acc_row(i, g)) ? dp[i] : 0.f;
                }
                ds[2 * h] = op_of<T>(dp, 0);
                ds[2 * h + 1] = op_of<T>(dp, 1);
            }
        }
        if (found) {
            if (!idle) {
                f32x16 add[DT];
                special_sums<T, D, BK>(add, col_base + tk, seen, g, true);
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) dq[dt] += add[dt];
            }
            __syncthreads();
            clear_special<T, BYTES, NW * 64>(tk, tid);
            __syncthreads();
        }
        if (!idle) {
            const Lds ck = opaque(col_base + tk);
#pragma unroll
            for (int c = 0; c < BK / 16; ++c)
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) mma(dq[dt], L::col_op(ck, 16 * c, dt), ds[c]);
        }
    }
    if ((lane & 31) >= rows) return;
    store_column<T, D>(reinterpret_cast<T*>(a.dq) + ((w.s.q0 + mine + (lane & 31)) * p.heads + head) * D, dq, p.scale, g);
}

template <typename T, int D>
hipError_t run_bwd(const BwdParams& b, hipStream_t stream) {
    const int share = b.p.heads / b.p.groups;
    if (b.tokens > 0) {
        const dim3 grid((unsigned)((b.tokens + kStatTokens - 1) / kStatTokens), (unsigned)((b.p.heads + kStatHeads - 1) / kStatHeads));
        hipLaunchKernelGGL((stats_kernel<T, D>), grid, dim3(256), 0, stream, b);
    }
    {
        BwdParams x = b;
        const int64_t grid = deal(&x.p, x.p.tk, 128, 1);
        if (grid < 0) return hipErrorInvalidValue;
        if (grid > 0) hipLaunchKernelGGL((dkv_kernel<T, D, 4>), dim3((unsigned)grid), dim3(256), 0, stream, x);
    }
    {
        BwdParams x = b;
        const int64_t grid = deal(&x.p, x.p.tq, 128, share);
        if (grid < 0) return hipErrorInvalidValue;
        if (grid > 0) hipLaunchKernelGGL((dq_kernel<T, D, 4>), dim3((unsigned)grid), dim3(256), 0, stream, x);
    }
    return hipGetLastError();
}

}  // namespace attn

hipError_t launch_attn_bwd(const AttnArgs& a) {
    const attn::BwdParams b{(const char*)a.q, (const char*)a.k, (const char*)a.v, (const char*)a.o, (const char*)a.d_o, a.lse,
                            a.dq, a.dk, a.dv, (float2*)a.stats, a.cu_q ? a.T : a.N * a.T, attn_shape(a)};
    const hipStream_t s = (hipStream_t)a.stream;
    if (a.dtype_bf16) return a.d == 64 ? attn::run_bwd<bf16, 64>(b, s) : attn::run_bwd<bf16, 128>(b, s);
    return a.d == 64 ? attn::run_bwd<float, 64>(b, s) : attn::run_bwd<float, 128>(b, s);
}

}  // namespace gdn2
