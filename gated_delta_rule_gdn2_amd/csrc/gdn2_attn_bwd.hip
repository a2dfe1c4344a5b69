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

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

// zero times x, added to `sum`: a NaN once anything was not finite
__device__ __forceinline__ float watch(float sum, float x) { return __builtin_fmaf(x, 0.f, sum); }

// A tile for which something is not finite, for 32 keys: what the mask hides is left out value by value.
// A query that is not finite has made its dS a NaN where it sees the key, so its own product takes the
// finite part; d_o adds to dv what is not finite in it.
template <typename T, int D>
__device__ __forceinline__ void special_dkv(f32x16 (&dk)[D / 32], f32x16 (&dv)[D / 32], const f32x16& s, const f32x16& dp, Lds tile,
                                            Seen seen, float scale_log2, int lane) {
    typedef Tile<T, D> L;
    constexpr int BYTES = kQueries * L::kRow;
    const int g = lane >> 5;
    const Lds cq = L::col_base(lane) + tile, co = cq + BYTES, ts = tile + 2 * BYTES;
    f32x16 p, ds;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int row = acc_row(i, g);
        const float lse = lds_get<float>(ts + row * 8), delta = lds_get<float>(ts + row * 8 + 4);
        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], scale_log2, -lse));
        p[i] = seen(row) ? x : 0.f;
        ds[i] = seen(row) ? x * (dp[i] - delta) : 0.f;
    }
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) {
        const f32x16 add = special_sum<T, D, kQueries>(co, dt, seen, g, false);
#pragma unroll
        for (int c = 0; c < kQueries / 16; ++c) {
            mma(dv[dt], finite_part<T>(L::col_op(co, 16 * c, dt)), op_of<T>(p, c));
            mma(dk[dt], finite_part<T>(L::col_op(cq, 16 * c, dt)), op_of<T>(ds, c));
        }
        dv[dt] += add;
    }
}

// A workgroup takes NW * KW * 32 keys of one key head, a wave KW blocks of 32; the queries that see them
// come by in tiles, the heads that share them one after the other.  S = Q K^T and dP = d_O V^T are formed with
// queries in the rows, so that P and dS are the next products' operands as they stand (dV^T = d_O^T P,
// dK^T = Q^T dS).  VL: values wait in LDS instead of registers.
template <typename T, int D, int NW, int KW, bool VL, int WAVES>
__global__ __launch_bounds__(NW * 64, WAVES) void dkv_kernel(BwdParams a) {
    typedef Tile<T, D> L;
    constexpr int KS = D / 16, DT = D / 32, BN = NW * KW * 32, BQ = kQueries, BYTES = BQ * L::kRow, STAGE = 2 * BYTES + 1024;
    __shared__ __attribute__((aligned(1024))) char lds[2 * STAGE + (VL ? BN * L::kRow : 0)];
    __shared__ int any_again;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Shape& p = a.p;
    Work w;
    if (!find_work(p, BN, 1, false, true, lane, &w)) return;
    w = uniform(w);
    const int kv = w.head, share = p.heads / p.groups, lq = w.s.lq, lk = w.s.lk;
    const int first = w.block * BN, mine = first + wave * KW * 32, rows = min(KW * 32, lk - mine);
    const int64_t off = (int64_t)lk - lq;  // where query 0 stands

    // the wave's keys and values; a lane's own are columns l % 32
    Op<T> k[KW][KS], v[VL ? 1 : KW][VL ? 1 : KS];
    if constexpr (VL)
        L::template stage<BN, NW>(lds_of(lds) + 2 * STAGE, a.v + (w.s.k0 + first) * p.v_stride + (int64_t)kv * L::kRow,
                                  span(min(BN, lk - first), p.v_stride, L::kRow), p.v_stride, wave, lane);
    {
        const auto rk = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(a.k + (w.s.k0 + mine) * p.k_stride + (int64_t)kv * L::kRow), 0,
                                                          span(rows, p.k_stride, L::kRow), 0x00020000);
        const auto rv = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(a.v + (w.s.k0 + mine) * p.v_stride + (int64_t)kv * L::kRow), 0,
                                                          span(rows, p.v_stride, L::kRow), 0x00020000);
#pragma unroll
        for (int j = 0; j < KW; ++j)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                k[j][ks] = global_op<T>(rk, (32 * j + (lane & 31)) * p.k_stride, ks, g);
                if constexpr (!VL) v[j][ks] = global_op<T>(rv, (32 * j + (lane & 31)) * p.v_stride, ks, g);
            }
    }
    if (tid == 0) any_again = 0;
    f32x16 dk[KW][DT], dv[KW][DT];
#pragma unroll
    for (int j = 0; j < KW; ++j)
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) dk[j][dt] = dv[j][dt] = zero16();

    // tiles of the queries that see some key of the block; the heads one after the other
    const int64_t from = first - off, to = min((int64_t)first + BN, (int64_t)lk) - 1 - off + p.window;  // [from, to)
    const int t0 = from > 0 ? (int)(min(from, (int64_t)lq) / BQ) : 0;
    const int t1 = to > 0 ? (int)((min(to, (int64_t)lq) + BQ - 1) / BQ) : 0;
    const uint32_t o_stride = (uint32_t)p.heads * L::kRow;
    const Lds base = lds_of(lds), row_base = L::row_base(lane), col_base = L::col_base(lane);
    const Lds tv = base + 2 * STAGE + wave * KW * 32 * L::kRow;  // the wave's values
    auto stage = [&](int h, int t, int buf) {
        const int head = kv * share + h, left = min(BQ, lq - t * BQ);
        const int64_t token = w.s.q0 + (int64_t)t * BQ;
        const Lds at = base + buf * STAGE;
        L::template stage<BQ, NW>(at, a.q + token * p.q_stride + (int64_t)head * L::kRow, span(left, p.q_stride, L::kRow), p.q_stride, wave, lane);
        L::template stage<BQ, NW>(at + BYTES, a.d_o + token * o_stride + (int64_t)head * L::kRow, span(left, o_stride, L::kRow), o_stride, wave, lane);
        if (wave == 0) load_words_to_lds(at + 2 * BYTES, rsrc_words(a.stats + (int64_t)head * a.tokens + token, left * 8), lane * 4);
    };
    const int count = t1 > t0 ? share * (t1 - t0) : 0;
    // Every tile that has to do with the wave's keys: f(its LDS, the place of its first query, its queries,
    // whether some query of it does not see some of the keys, or is none).
    auto walk = [&](auto f) {
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
            const int64_t place = off + (int64_t)t * BQ;
            const int left = lq - t * BQ;
            h = next_h;
            t = next_t;
            if (rows <= 0 || place + BQ - 1 < mine || place > (int64_t)mine + KW * 32 - 2 + p.window) continue;
            f(base + (n & 1) * STAGE, place, left,
              place < (int64_t)mine + KW * 32 - 1 || place + BQ - 1 >= (int64_t)mine + p.window || left < BQ);
        }
    };
    f32x16 s[KW], dp[KW];
    auto scores = [&](Lds tq) {
        const Lds rq = opaque(row_base + tq), ro = opaque(row_base + tq + BYTES), rv = VL ? opaque(row_base + tv) : 0;
#pragma unroll
        for (int j = 0; j < KW; ++j) s[j] = dp[j] = zero16();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const Op<T> x = L::row_op(rq, 0, ks);
#pragma unroll
            for (int j = 0; j < KW; ++j) mma(s[j], x, k[j][ks]);
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const Op<T> x = L::row_op(ro, 0, ks);
#pragma unroll
            for (int j = 0; j < KW; ++j) {
                if constexpr (VL) mma(dp[j], x, L::row_op(rv, 32 * j, ks));
                else mma(dp[j], x, v[j][ks]);
            }
        }
    };
    // the queries of a tile that see the lane's key of block j
    auto seen_by = [&](int j, int64_t place, int left) {
        const int64_t lo = (int64_t)mine + 32 * j + (lane & 31) - place, hi = min(lo + p.window - 1, (int64_t)left - 1);
        return seen_between((int)min(max(lo, (int64_t)-1), (int64_t)BQ), (int)max((int64_t)-2, min(hi, (int64_t)BQ)));
    };
    // whether anything of a tile is not finite: it is then in S, dP, lse or delta
    auto special = [&](Lds tq) {
        float sum = watch(0.f, lds_get<float>(tq + 2 * BYTES + lane * 4));
#pragma unroll
        for (int j = 0; j < KW; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) sum = watch(watch(sum, s[j][i]), dp[j][i]);
        return __any(sum != 0.f);
    };
    bool again = false;
    // FIRST: a tile with something that is not finite is left to a second walk over all of them
    auto tile = [&](auto FIRST, Lds tq, int64_t place, int left, bool cut) {
        scores(tq);
        if (cut) {
            if (special(tq)) {
                if constexpr (FIRST.value) {
                    again = true;
                } else {
#pragma unroll
                    for (int j = 0; j < KW; ++j)
                        special_dkv<T, D>(dk[j], dv[j], s[j], dp[j], tq, seen_by(j, place, left), p.scale_log2, lane);
                }
                return;
            }
#pragma unroll
            for (int j = 0; j < KW; ++j) {
                const Seen seen = seen_by(j, place, left);
#pragma unroll
                for (int i = 0; i < 16; ++i) s[j][i] = seen(acc_row(i, g)) ? s[j][i] : -__builtin_inff();
            }
        }
        const Lds ts = tq + 2 * BYTES;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const f32x4 x = lds_get<f32x4>(ts + (8 * c + 4 * g) * 8), y = lds_get<f32x4>(ts + (8 * c + 4 * g) * 8 + 16);
            const float lse[4] = {x[0], x[2], y[0], y[2]}, delta[4] = {x[1], x[3], y[1], y[3]};
#pragma unroll
            for (int j = 0; j < KW; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 4 * c + e;
                    s[j][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][i], p.scale_log2, -lse[e]));
                    dp[j][i] = s[j][i] * (dp[j][i] - delta[e]);
                }
        }
        Op<T> pr[KW][BQ / 16], ds[KW][BQ / 16];
#pragma unroll
        for (int j = 0; j < KW; ++j)
#pragma unroll
            for (int c = 0; c < BQ / 16; ++c) {
                pr[j][c] = op_of<T>(s[j], c);
                ds[j][c] = op_of<T>(dp[j], c);
            }
        const Lds cq = opaque(col_base + tq), co = opaque(col_base + tq + BYTES);
#pragma unroll
        for (int c = 0; c < BQ / 16; ++c)
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                const Op<T> x = L::col_op(co, 16 * c, dt), y = L::col_op(cq, 16 * c, dt);
#pragma unroll
                for (int j = 0; j < KW; ++j) {
                    mma(dv[j][dt], x, pr[j][c]);
                    mma(dk[j][dt], y, ds[j][c]);
                }
            }
    };
    walk([&](Lds tq, int64_t place, int left, bool cut) { tile(Yes{}, tq, place, left, cut); });
    if (again) any_again = 1;
    __syncthreads();
    if (any_again) {
        if (again) {
#pragma unroll
            for (int j = 0; j < KW; ++j)
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) dk[j][dt] = dv[j][dt] = zero16();
        }
        walk([&](Lds tq, int64_t place, int left, bool cut) {
            if (again) tile(No{}, tq, place, left, cut);
        });
    }
#pragma unroll
    for (int j = 0; j < KW; ++j) {
        if (32 * j + (lane & 31) >= rows) continue;
        const int64_t at = ((w.s.k0 + mine + 32 * j + (lane & 31)) * p.groups + kv) * D;
        store_column<T, D>(reinterpret_cast<T*>(a.dk) + at, dk[j], p.scale, g);
        store_column<T, D>(reinterpret_cast<T*>(a.dv) + at, dv[j], 1.f, g);
    }
}

// ---- dq ---------------------------------------------------------------------------------------

template <typename T> constexpr int kKeys = sizeof(T) == 2 ? 64 : 32;  // keys in a tile

// A workgroup takes 32 queries of one head a wave; keys and values come by in tiles.  S^T = K Q^T and
// dP^T = V d_O^T have keys in the rows, so that dS is the next product's operand (dQ^T = K^T dS^T).
template <typename T, int D, int NW>
__global__ __launch_bounds__(NW * 64, D * sizeof(T) > 256 ? 1 : 2) void dq_kernel(BwdParams a) {
    typedef Tile<T, D> L;
    constexpr int BK = kKeys<T>, KS = D / 16, DT = D / 32, BM = NW * 32, BYTES = BK * L::kRow;
    __shared__ __attribute__((aligned(1024))) char lds[2 * 2 * BYTES];
    __shared__ int any_again;
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
    if (tid == 0) any_again = 0;
    // every tile that the wave's queries see something of: f(its LDS, its first key, whether not all of it)
    auto walk = [&](auto f) {
        if (t0 < t1) stage(t0);
        for (int t = t0; t < t1; ++t) {
            tile_barrier();
            if (t + 1 < t1) stage(t + 1);
            const int key0 = t * BK;
            if (rows <= 0 || key0 > pos0 + rows - 1 || key0 + BK - 1 <= pos0 - p.window) continue;
            f(base + (t & 1) * 2 * BYTES, key0, key0 + BK - 1 > pos0 || key0 <= pos0 + 31 - p.window);
        }
    };
    // S^T and dP^T of 32 keys
    f32x16 s, dp;
    auto scores = [&](Lds rk, Lds rv, int h) {
        s = dp = zero16();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) mma(s, L::row_op(rk, 32 * h, ks), q[ks]);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) mma(dp, L::row_op(rv, 32 * h, ks), d_o[ks]);
    };
    // whether anything that meets there is not finite
    const float bad = watch(watch(0.f, lse), delta);
    auto special = [&] {
        float sum = bad;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum = watch(watch(sum, s[i]), dp[i]);
        return __any(sum != 0.f);
    };
    bool again = false;
    // FIRST: a tile with something that is not finite is left to a second walk over all of them, where what
    // the mask hides is left out value by value and a key that is not finite makes what sees it a NaN
    auto tile = [&](auto FIRST, Lds tk, int key0, bool cut) {
        const Lds rk = opaque(row_base + tk), rv = opaque(row_base + tk + BYTES);
        const Seen seen = seen_between(pos - key0 - p.window + 1, pos - key0);
        Op<T> ds[BK / 16];
        bool left = false;
#pragma unroll
        for (int h = 0; h < BK / 32; ++h) {
            scores(rk, rv, h);
            if (cut) {
                left = left || special();
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = seen(32 * h + acc_row(i, g)) ? s[i] : -__builtin_inff();
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], p.scale_log2, -lse)) * (dp[i] - delta);
                dp[i] = FIRST.value || !cut || seen(32 * h + acc_row(i, g)) ? x : 0.f;
            }
            ds[2 * h] = op_of<T>(dp, 0);
            ds[2 * h + 1] = op_of<T>(dp, 1);
        }
        if (FIRST.value && left) {
            again = true;
            return;
        }
        const Lds ck = opaque(col_base + tk);
        if (left) {
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                const f32x16 add = special_sum<T, D, BK>(ck, dt, seen, g, true);
#pragma unroll
                for (int c = 0; c < BK / 16; ++c) mma(dq[dt], finite_part<T>(L::col_op(ck, 16 * c, dt)), ds[c]);
                dq[dt] += add;
            }
            return;
        }
#pragma unroll
        for (int c = 0; c < BK / 16; ++c)
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) mma(dq[dt], L::col_op(ck, 16 * c, dt), ds[c]);
    };
    walk([&](Lds tk, int key0, bool cut) { tile(Yes{}, tk, key0, cut); });
    if (again) any_again = 1;
    __syncthreads();
    if (any_again) {
        if (again) {
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) dq[dt] = zero16();
        }
        walk([&](Lds tk, int key0, bool cut) {
            if (again) tile(No{}, tk, key0, cut);
        });
    }
    if ((lane & 31) >= rows) return;
    store_column<T, D>(reinterpret_cast<T*>(a.dq) + ((w.s.q0 + mine + (lane & 31)) * p.heads + head) * D, dq, p.scale, g);
}

#ifndef KWT
#define KWT 1
#endif
template <typename T, int D>
hipError_t run_bwd(const BwdParams& b, hipStream_t stream) {
    const int share = b.p.heads / b.p.groups;
    if (b.tokens > 0) {
        const dim3 grid((unsigned)((b.tokens + kStatTokens - 1) / kStatTokens), (unsigned)((b.p.heads + kStatHeads - 1) / kStatHeads));
        hipLaunchKernelGGL((stats_kernel<T, D>), grid, dim3(256), 0, stream, b);
    }
    {
        BwdParams x = b;
        constexpr bool wide = D * sizeof(T) == 256 && KWT == 2;
        constexpr int KW = wide ? 2 : 1;
        const int64_t grid = deal(&x.p, x.p.tk, 128 * KW, 1);
        if (grid < 0) return hipErrorInvalidValue;
        if (grid > 0)
            hipLaunchKernelGGL((dkv_kernel<T, D, 4, KW, D * sizeof(T) == 256, (D * sizeof(T) > 256 || wide) ? 1 : 2>), dim3((unsigned)grid), dim3(256), 0, stream, x);
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
