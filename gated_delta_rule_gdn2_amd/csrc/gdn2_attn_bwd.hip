// gdn2_attn_bwd.hip -- gradients of causal attention, which forms the probabilities again.
//
//   P_ij = e^(scale q_i . k_j - lse_i) for the keys j that query i sees (0 for the others),
//   delta_i = d_o_i . o_i,  dP_ij = d_o_i . v_j,  dS_ij = P_ij (dP_ij - delta_i),
//   dv_j = sum_i P_ij d_o_i,  dk_j = scale sum_i dS_ij q_i,  dq_i = scale sum_j dS_ij k_j,
// the sums over i also over the query heads that share a key head.
//
// Two kernels: one workgroup a block of queries for dq, which also leaves lse in base 2 and -delta of its
// queries in the workspace, then one a block of keys for dk and dv.  Every sum is formed by one wave in a fixed
// order: equal calls give equal bits, at the price of S and dP twice (7 products instead of 5; partial sums of
// dq for each block of keys would move more bytes than that takes).  Sums are fp32; with bf16 inputs P and dS
// are rounded to bf16 once, as the matrix unit's operands, and gradients on the store.
//
// At 8 x 4096 tokens, 16 heads of 128 sharing 8, window 2048, bf16: dq 590 to 640 us, dk and dv 740 to 820,
// matrix units busy for 50 to 56% of the cycles at 1.5 to 1.8 GHz (980 to 1050 TFLOP/s of the 7 products).  Heads of
// 64 are bound by vector issue, three waves a SIMD (8 x 4096 tokens of 16 heads: 1000 us in all).  fp32: 2 x 4096
// tokens, 16 heads of 128 sharing 4, 5.0 ms (96 TFLOP/s of the 7 products), of 64 2.16 ms (111).
//
// A product multiplies what a query does not see by zero, which infinities and NaN survive.  A wave that meets
// a value that is not finite in a tile that the mask cuts gives up, and its workgroup starts again in a form
// that leaves out value by value what the mask hides.
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
    float* lse2;      // [heads][tokens]: lse in base 2
    float* no_delta;  // [heads][tokens]: -delta, what dP starts from
    int64_t tokens;   // queries in all
    float* parts;     // of more than one part: [part][dk, dv][keys][key heads][d], unscaled
    int64_t keys;     // keys in all
    Shape p;
};

// ---- dq ---------------------------------------------------------------------------------------

template <typename T, int SW> constexpr int kKeys = sizeof(T) == 2 && SW == 1 ? 64 : 32;  // keys in a tile
template <typename T, int D, int SW> constexpr int kDqLds = SW * 2 * 2 * kKeys<T, SW> * Tile<T, D>::kRow;

// A workgroup takes 32 queries of one head a wave; keys and values come by in tiles.  S^T = K Q^T and
// dP^T = V d_O^T have keys in the rows, so that dS is the next product's operand (dQ^T = K^T dS^T).
// SW > 1: all waves share 32 queries; each takes every SWth tile of keys, with tiles of its own in LDS, and
// their sums are joined at the end.  Returns whether some wave gave up; it has written nothing then.
template <typename T, int D, int NW, int SW, bool FIRST>
__device__ __forceinline__ bool dq_block(const BwdParams& a, Lds base, int* flag) {
    typedef Tile<T, D> L;
    static_assert(SW == 1 || SW == NW, "each wave its own queries, or all the same");
    constexpr int BK = kKeys<T, SW>, KS = D / 16, DT = D / 32, BM = NW / SW * 32, BYTES = BK * L::kRow;
    const int lane = threadIdx.x & 63, g = lane >> 5;
    const int all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = SW == 1 ? all_waves : 0, part = SW == 1 ? 0 : all_waves;
    const Shape& p = a.p;
    Work w;
    if (!find_work(p, BM, p.heads / p.groups, true, false, lane, &w)) return false;
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

    const Lds row_base = L::row_base(lane), col_base = L::col_base(lane);
    auto place = [&](int t) { return base + (part * 2 + (t / SW & 1)) * 2 * BYTES; };
    auto stage = [&](int t) {
        const Lds at = place(t);
        const int left = min(BK, lk - t * BK);
        L::template stage<BK, NW / SW>(at, kp + (int64_t)t * BK * p.k_stride, span(left, p.k_stride, L::kRow), p.k_stride, wave, lane);
        L::template stage<BK, NW / SW>(at + BYTES, vp + (int64_t)t * BK * p.v_stride, span(left, p.v_stride, L::kRow), p.v_stride, wave, lane);
    };
    // queries, d_o and o: by way of the tiles' places in LDS, if they have room there, so that rows are read whole
    constexpr bool VIA = BM * L::kRow <= 2 * BYTES;
    const int64_t row0 = (w.s.q0 + first) * p.heads + head;
    const char* qp = a.q + (w.s.q0 + first) * p.q_stride + (int64_t)head * L::kRow;
    const uint32_t q_span = span(min(BM, lq - first), p.q_stride, L::kRow), o_span = span(min(BM, lq - first), o_stride, L::kRow);
    Op<T> q[KS], d_o[KS];
    float delta = 0.f;
    auto dot = [&](const Op<T>& x, const Op<T>& y) {
#pragma unroll
        for (int e = 0; e < 8; ++e) delta = __builtin_fmaf(to_f32((T)x.v[e]), to_f32((T)y.v[e]), delta);
    };
    if constexpr (VIA) {
        // (of the first wave, where waves have tiles of their own)
        const Lds one = base + (t0 / SW & 1) * 2 * BYTES, two = base + (~(t0 / SW) & 1) * 2 * BYTES, own = row_base + wave * 32 * L::kRow;
        L::template stage<BM, NW>(one, qp, q_span, p.q_stride, all_waves, lane);
        L::template stage<BM, NW>(two, a.d_o + row0 * L::kRow, o_span, o_stride, all_waves, lane);
        tile_barrier();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            q[ks] = L::row_op(own + one, 0, ks);
            d_o[ks] = L::row_op(own + two, 0, ks);
        }
        lds_barrier();
        if (t0 + part < t1) stage(t0 + part);
        L::template stage<BM, NW>(two, a.o + row0 * L::kRow, o_span, o_stride, all_waves, lane);
        tile_barrier();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) dot(d_o[ks], L::row_op(own + two, 0, ks));
        if (SW > 1) lds_barrier();
    } else {
        const auto rq = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(qp), 0, q_span, 0x00020000);
        const auto rd = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(a.d_o + row0 * L::kRow), 0, o_span, 0x00020000);
        const auto ro = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(a.o + row0 * L::kRow), 0, o_span, 0x00020000);
        const uint32_t row = wave * 32 + (lane & 31);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            q[ks] = global_op<T>(rq, row * p.q_stride, ks, g);
            d_o[ks] = global_op<T>(rd, row * o_stride, ks, g);
            dot(d_o[ks], global_op<T>(ro, row * o_stride, ks, g));
        }
        if (t0 + part < t1) stage(t0 + part);
    }
    delta += other_half(delta, lane);
    float lse = 0.f;
    if ((lane & 31) < rows) {
        lse = a.lse[row0 + (int64_t)(wave * 32 + (lane & 31)) * p.heads] * kLog2e;
        const int64_t at = (int64_t)head * a.tokens + w.s.q0 + mine + (lane & 31);
        if (part == 0 && g == 0) a.lse2[at] = lse;
        if (part == 0 && g == 1) a.no_delta[at] = -delta;
    }
    f32x16 dq[DT];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) dq[dt] = zero16();
    bool again = false;
    for (int t = t0 + part; t < t1; t += SW) {
        if (SW == 1) tile_barrier();
        else own_tile_wait();
        if (t + SW < t1) stage(t + SW);
        const int key0 = t * BK;
        if (rows <= 0 || key0 > pos0 + rows - 1 || key0 + BK - 1 <= pos0 - p.window) continue;  // nothing that the wave's queries see
        const bool cut = key0 + BK - 1 > pos0 || key0 <= pos0 + 31 - p.window;                 // not all that they see
        const Lds tk = place(t), rk = opaque(row_base + tk), rv = opaque(row_base + tk + BYTES);
        const Seen seen = seen_between(pos - key0 - p.window + 1, pos - key0);  // the lane's query's
        Op<T> ds[BK / 16];
        float sum = watch(watch(0.f, lse), delta);
#pragma unroll
        for (int h = 0; h < BK / 32; ++h) {
            f32x16 s = zero16(), dp = zero16();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) mma(s, L::row_op(rk, 32 * h, ks), q[ks]);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) mma(dp, L::row_op(rv, 32 * h, ks), d_o[ks]);
            if (cut) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    sum = watch(watch(sum, s[i]), dp[i]);
                    s[i] = seen(32 * h + acc_row(i, g)) ? s[i] : -__builtin_inff();
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], p.scale_log2, -lse)) * (dp[i] - delta);
                dp[i] = FIRST || !cut || seen(32 * h + acc_row(i, g)) ? x : 0.f;
            }
            ds[2 * h] = op_of<T>(dp, 0);
            ds[2 * h + 1] = op_of<T>(dp, 1);
        }
        const Lds ck = opaque(col_base + tk);
        if (FIRST && cut) again = again || __any(sum != 0.f);
        if (!FIRST && cut) {  // a key that is not finite makes what sees it a NaN
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                const f32x16 add = special_sum<T, D, BK>(ck, dt, seen, g, true);
#pragma unroll
                for (int c = 0; c < BK / 16; ++c) mma(dq[dt], finite_part<T>(L::col_op(ck, 16 * c, dt)), ds[c]);
                dq[dt] += add;
            }
            continue;
        }
#pragma unroll
        for (int c = 0; c < BK / 16; ++c)
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) mma(dq[dt], L::col_op(ck, 16 * c, dt), ds[c]);
    }
    if (FIRST && again) *flag = 1;
    lds_barrier();
    const bool any = FIRST && *flag != 0;
    if constexpr (SW > 1) {
        if (any) return any;
        static_assert(WaveSums<D, SW>::kBytes <= kDqLds<T, D, SW>, "room for the sums");
        WaveSums<D, SW> sums;
        sums.add(base, dq, p.scale, part, lane);
        if ((lane & 31) < rows) sums.template store<T>((T*)a.dq + (row0 + (int64_t)(lane & 31) * p.heads) * D, 1.f, part, g);
        return any;
    }
    if (rows > 0 && !again)
        store_rows<T, D>(base + wave * 32 * L::kRow, (char*)a.dq + (row0 + (int64_t)wave * 32 * p.heads) * L::kRow, o_stride, rows, dq, p.scale, lane);
    return any;
}
// a call of its own, so that the kernel keeps its registers to the first form
template <typename T, int D, int NW, int SW>
__device__ __attribute__((noinline)) void dq_again(BwdParams a, Lds base) {
    dq_block<T, D, NW, SW, false>(a, base, nullptr);
}

template <typename T, int D, int NW, int SW>
__global__ __launch_bounds__(NW * 64, SW > 1 ? (kDqLds<T, D, SW> > 80000 ? 1 : 2) : D == 64 ? 3 : sizeof(T) == 4 ? 1 : 2)
void dq_kernel(BwdParams a) {
    __shared__ __attribute__((aligned(1024))) char lds[kDqLds<T, D, SW>];
    __shared__ int flag;
    if (threadIdx.x == 0) flag = 0;
    if (dq_block<T, D, NW, SW, true>(a, lds_of(lds), &flag)) {
        __syncthreads();
        dq_again<T, D, NW, SW>(a, lds_of(lds));
    }
}

// ---- dk and dv --------------------------------------------------------------------------------

// Queries in a tile: at 64 channels of bf16 two blocks of 32, which share the loop's own instructions (8 x 4096
// tokens, 16 heads: 1033 us for all gradients, 1052 with one).
template <typename T, int D, int SW> constexpr int kQueries = D * sizeof(T) == 128 && SW == 1 ? 64 : 32;
// LDS of a tile: queries, d_o, and of each lse in base 2 and -delta; and of the whole workgroup
template <typename T, int D, int SW> constexpr int kStage = 2 * kQueries<T, D, SW> * Tile<T, D>::kRow + 1024;
template <typename T, int D, int NW, int SW> constexpr int kDkvLds = SW * 2 * kStage<T, D, SW> + NW / SW * 32 * Tile<T, D>::kRow;

// A workgroup takes NW * 32 keys of one key head, a wave 32; the queries that see them come by in tiles, the
// heads that share them one after the other.  S = Q K^T and dP = d_O V^T have queries in the rows, so that P and
// dS are the next products' operands as they stand (dV^T = d_O^T P, dK^T = Q^T dS).  Keys stay in registers,
// values in LDS: with both in registers there is one wave a SIMD, which took 1.65 ms at the shape above, against
// 0.75 ms.
// SW > 1: all waves share 32 keys; each takes every SWth tile of queries, as in dq_block.
template <typename T, int D, int NW, int SW, bool FIRST>
__device__ __forceinline__ bool dkv_block(const BwdParams& a, Lds base, int* flag) {
    typedef Tile<T, D> L;
    static_assert(SW == 1 || SW == NW, "each wave its own keys, or all the same");
    constexpr int KS = D / 16, DT = D / 32, BN = NW / SW * 32, BQ = kQueries<T, D, SW>, BYTES = BQ * L::kRow, STAGE = kStage<T, D, SW>;
    const int lane = threadIdx.x & 63, g = lane >> 5;
    const int all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = SW == 1 ? all_waves : 0, part = SW == 1 ? 0 : all_waves;
    const Shape& p = a.p;
    Work w;
    if (!find_work(p, BN, 1, false, true, lane, &w)) return false;
    w = uniform(w);
    const int kv = w.head, share = p.heads / p.groups, lq = w.s.lq, lk = w.s.lk;
    const int first = w.block * BN, mine = first + wave * 32, rows = min(32, lk - mine);
    const int64_t off = (int64_t)lk - lq;  // where query 0 stands

    const Lds row_base = L::row_base(lane), col_base = L::col_base(lane), tv = base + SW * 2 * STAGE;
    // keys come by way of the tiles' places in LDS
    Op<T> k[KS];
    {
        const int left = min(BN, lk - first);
        static_assert(BN * L::kRow <= 2 * STAGE, "room for the keys");
        L::template stage<BN, NW>(base, a.k + (w.s.k0 + first) * p.k_stride + (int64_t)kv * L::kRow, span(left, p.k_stride, L::kRow), p.k_stride, all_waves, lane);
        L::template stage<BN, NW>(tv, a.v + (w.s.k0 + first) * p.v_stride + (int64_t)kv * L::kRow, span(left, p.v_stride, L::kRow), p.v_stride, all_waves, lane);
        tile_barrier();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) k[ks] = L::row_op(row_base + base + wave * 32 * L::kRow, 0, ks);
        lds_barrier();
    }
    f32x16 dk[DT], dv[DT];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) dk[dt] = dv[dt] = zero16();

    // tiles of the queries that see some key of the block; the heads one after the other
    const int64_t from = first - off, to = min((int64_t)first + BN, (int64_t)lk) - 1 - off + p.window;  // [from, to)
    const int t0 = from > 0 ? (int)(min(from, (int64_t)lq) / BQ) : 0;
    const int t1 = to > 0 ? (int)((min(to, (int64_t)lq) + BQ - 1) / BQ) : 0;
    const uint32_t o_stride = (uint32_t)p.heads * L::kRow;
    auto stage = [&](int h, int t, int buf) {
        const int head = kv * share + h, left = min(BQ, lq - t * BQ);
        const int64_t token = w.s.q0 + (int64_t)t * BQ;
        const Lds at = base + (part * 2 + buf) * STAGE;
        L::template stage<BQ, NW / SW>(at, a.q + token * p.q_stride + (int64_t)head * L::kRow, span(left, p.q_stride, L::kRow), p.q_stride, wave, lane);
        L::template stage<BQ, NW / SW>(at + BYTES, a.d_o + token * o_stride + (int64_t)head * L::kRow, span(left, o_stride, L::kRow), o_stride, wave, lane);
        if (wave == 0) {  // rows that are none repeat the last
            const int64_t from = (int64_t)head * a.tokens + token;
            if constexpr (BQ == 32) {
                load_far_words_to_lds(at + 2 * BYTES, (g ? a.no_delta : a.lse2) + from + min(lane & 31, left - 1));
            } else {
                load_far_words_to_lds(at + 2 * BYTES, a.lse2 + from + min(lane, left - 1));
                load_far_words_to_lds(at + 2 * BYTES + 256, a.no_delta + from + min(lane, left - 1));
            }
        }
    };
    // the workgroup's part of them
    const int all = t1 > t0 ? share * (t1 - t0) : 0, per = (all + (int)gridDim.y - 1) / (int)gridDim.y;
    const int n0 = min(per * (int)blockIdx.y, all) + part, count = min(n0 - part + per, all);
    int h = 0, t = t0;
    auto after = [&](int steps) {  // `steps` tiles on
        t += steps;
        while (t >= t1) {
            t -= t1 - t0;
            ++h;
        }
    };
    bool again = false;
    if (n0 < count) {
        after(n0);
        stage(h, t, 0);
    }
    for (int n = n0; n < count; n += SW) {
        if (SW == 1) tile_barrier();
        else own_tile_wait();
        const int64_t place0 = off + (int64_t)t * BQ;  // of the tile's first query
        const int left0 = lq - t * BQ;                 // its queries
        const Lds tile = base + (part * 2 + ((n - n0) / SW & 1)) * STAGE;
        if (n + SW < count) {
            after(SW);
            stage(h, t, ((n - n0) / SW + 1) & 1);
        }
#pragma unroll
        for (int u = 0; u < BQ / 32; ++u) {
            const int64_t place = place0 + 32 * u;
            const int left = left0 - 32 * u;
            // no query of the block sees a key of the wave's; or some query does not see some key, or is none
            if (rows <= 0 || left <= 0 || place + 31 < mine || place > (int64_t)mine + 30 + p.window) continue;
            const bool cut = place < (int64_t)mine + 31 || place + 31 >= (int64_t)mine + p.window || left < 32;
            const Lds tq = tile + u * 32 * L::kRow, ts = tile + 2 * BYTES + u * 128 + 16 * g;
            const Lds rq = opaque(row_base + tq), ro = opaque(row_base + tq + BYTES), rv = opaque(row_base + tv + wave * 32 * L::kRow);
            f32x16 s = zero16(), dp;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const f32x4 x = lds_get<f32x4>(ts + BQ * 4 + 32 * c);
#pragma unroll
                for (int e = 0; e < 4; ++e) dp[4 * c + e] = x[e];
            }
            // the two chains of products side by side, operands two steps at a time (1466 and 1442 us at the shape above)
            constexpr int C = sizeof(T) == 2 ? 2 : 1;
#pragma unroll
            for (int k0 = 0; k0 < KS; k0 += C) {
                Op<T> xq[C], xo[C], xv[C];
#pragma unroll
                for (int ks = 0; ks < C; ++ks) {
                    xq[ks] = L::row_op(rq, 0, k0 + ks);
                    xo[ks] = L::row_op(ro, 0, k0 + ks);
                    xv[ks] = L::row_op(rv, 0, k0 + ks);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int ks = 0; ks < C; ++ks) {
                    mma(s, xq[ks], k[k0 + ks]);
                    mma(dp, xo[ks], xv[ks]);
                }
            }
            float lse[16];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const f32x4 x = lds_get<f32x4>(ts + 32 * c);
#pragma unroll
                for (int e = 0; e < 4; ++e) lse[4 * c + e] = x[e];
            }
            Seen seen{0, 32};  // the queries that see the lane's key
            if (cut) {
                const int64_t lo = (int64_t)mine + (lane & 31) - place, hi = min(lo + p.window - 1, (int64_t)left - 1);
                seen = seen_between((int)min(max(lo, (int64_t)-1), (int64_t)32), (int)max((int64_t)-2, min(hi, (int64_t)32)));
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    sum = watch(watch(watch(sum, s[i]), dp[i]), lse[i]);
                    s[i] = seen(acc_row(i, g)) ? s[i] : -__builtin_inff();
                }
                if (FIRST) again = again || __any(sum != 0.f);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], p.scale_log2, -lse[i]));
                dp[i] *= s[i];
            }
            if (!FIRST && cut) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const bool yes = seen(acc_row(i, g));
                    s[i] = yes ? s[i] : 0.f;
                    dp[i] = yes ? dp[i] : 0.f;
                }
            }
            Op<T> pr[2], ds[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                pr[c] = op_of<T>(s, c);
                ds[c] = op_of<T>(dp, c);
            }
            const Lds cq = opaque(col_base + tq), co = opaque(col_base + tq + BYTES);
            if (!FIRST && cut) {
                // a query that is not finite has made its dS a NaN where it sees the key, so its own product takes
                // the finite part; d_o adds to dv what is not finite in it
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) {
                    const f32x16 add = special_sum<T, D, 32>(co, dt, seen, g, false);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        mma(dv[dt], finite_part<T>(L::col_op(co, 16 * c, dt)), pr[c]);
                        mma(dk[dt], finite_part<T>(L::col_op(cq, 16 * c, dt)), ds[c]);
                    }
                    dv[dt] += add;
                }
                continue;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) {
                    mma(dv[dt], L::col_op(co, 16 * c, dt), pr[c]);
                    mma(dk[dt], L::col_op(cq, 16 * c, dt), ds[c]);
                }
        }
    }
    if (FIRST && again) *flag = 1;
    lds_barrier();
    const bool any = FIRST && *flag != 0;
    if constexpr (SW > 1) {
        if (any) return any;
        static_assert(WaveSums<D, SW>::kBytes <= kDkvLds<T, D, NW, SW>, "room for the sums");
        const int64_t at = ((w.s.k0 + mine + (lane & 31)) * p.groups + kv) * D, size = a.keys * p.groups * D;
        const bool whole = gridDim.y == 1, live = (lane & 31) < rows;
        float* parts = a.parts + 2 * blockIdx.y * size + at;
        WaveSums<D, SW> sums;
        sums.add(base, dk, whole ? p.scale : 1.f, part, lane);
        if (live && whole) sums.template store<T>((T*)a.dk + at, 1.f, part, g);
        else if (live) sums.template store<float>(parts, 1.f, part, g);
        lds_barrier();
        sums.add(base, dv, 1.f, part, lane);
        if (live && whole) sums.template store<T>((T*)a.dv + at, 1.f, part, g);
        else if (live) sums.template store<float>(parts + size, 1.f, part, g);
        return any;
    }
    if (rows > 0 && !again && gridDim.y > 1) {
        const int64_t size = a.keys * p.groups * D;
        float* parts = a.parts + 2 * blockIdx.y * size + ((w.s.k0 + mine + (lane & 31)) * p.groups + kv) * D;
        if ((lane & 31) < rows) {
            store_column<float, D>(parts, dk, 1.f, g);
            store_column<float, D>(parts + size, dv, 1.f, g);
        }
    } else if (rows > 0 && !again) {
        const int64_t at = ((w.s.k0 + mine) * p.groups + kv) * L::kRow, stride = (int64_t)p.groups * L::kRow;
        const Lds own = base + wave * 32 * L::kRow;
        store_rows<T, D>(own, (char*)a.dk + at, stride, rows, dk, p.scale, lane);
        __builtin_amdgcn_wave_barrier();
        store_rows<T, D>(own, (char*)a.dv + at, stride, rows, dv, 1.f, lane);
    }
    return any;
}
template <typename T, int D, int NW, int SW>
__device__ __attribute__((noinline)) void dkv_again(BwdParams a, Lds base) {
    dkv_block<T, D, NW, SW, false>(a, base, nullptr);
}

template <typename T, int D, int NW, int SW>
__global__ __launch_bounds__(NW * 64, SW > 1 ? (kDkvLds<T, D, NW, SW> > 80000 ? 1 : 2) : D * sizeof(T) > 256 ? 1 : D * sizeof(T) > 128 ? 2 : 3)
void dkv_kernel(BwdParams a) {
    __shared__ __attribute__((aligned(1024))) char lds[kDkvLds<T, D, NW, SW>];
    __shared__ int flag;
    if (threadIdx.x == 0) flag = 0;
    if (dkv_block<T, D, NW, SW, true>(a, lds_of(lds), &flag)) {
        __syncthreads();
        dkv_again<T, D, NW, SW>(a, lds_of(lds));
    }
}

// Joins the parts of dk and dv, in their order: D / 4 threads a row.
template <typename T, int D>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ parts, T* __restrict__ dk, T* __restrict__ dv,
                                                   float scale, int64_t rows, int splits, Owned owned) {
    const int64_t row = (int64_t)blockIdx.x * (1024 / D) + threadIdx.x / (D / 4);
    const int64_t at = row * D + threadIdx.x % (D / 4) * 4, size = rows * D;
    if (row >= rows || !owned_by_lane(owned, row / owned.heads)) return;
    f32x4 sk{0.f, 0.f, 0.f, 0.f}, sv = sk;
    for (int i = 0; i < splits; ++i) {
        sk += *reinterpret_cast<const f32x4*>(parts + 2 * i * size + at);
        sv += *reinterpret_cast<const f32x4*>(parts + (2 * i + 1) * size + at);
    }
    float a[4], b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        a[e] = sk[e] * scale;
        b[e] = sv[e];
    }
    store_vec_any<T, 4>(dk + at, a);
    store_vec_any<T, 4>(dv + at, b);
}

template <typename T, int D, int NW, int SW>
hipError_t run_dq(BwdParams x, hipStream_t stream) {
    const int64_t grid = deal(&x.p, x.p.tq, NW / SW * 32, x.p.heads / x.p.groups);
    if (grid < 0) return hipErrorInvalidValue;
    if (grid > 0) hipLaunchKernelGGL((dq_kernel<T, D, NW, SW>), dim3((unsigned)grid), dim3(NW * 64), 0, stream, x);
    return hipGetLastError();
}
template <typename T, int D, int NW, int SW>
hipError_t run_dkv(BwdParams x, int splits, hipStream_t stream) {
    const int64_t grid = deal(&x.p, x.p.tk, NW / SW * 32, 1);
    if (grid < 0) return hipErrorInvalidValue;
    if (grid == 0) return hipSuccess;
    hipLaunchKernelGGL((dkv_kernel<T, D, NW, SW>), dim3((unsigned)grid, (unsigned)splits), dim3(NW * 64), 0, stream, x);
    if (splits > 1) {
        const int64_t rows = x.keys * x.p.groups;
        hipLaunchKernelGGL((join_kernel<T, D>), dim3((unsigned)((rows + 1024 / D - 1) / (1024 / D))), dim3(256), 0, stream, x.parts,
                           (T*)x.dk, (T*)x.dv, x.p.scale, rows, splits, Owned{x.p.cu_k, x.p.n, x.p.tk, x.p.groups});
    }
    return hipGetLastError();
}

// How the backward pass is launched.  Workgroups whose waves share 32 queries or keys are four times as many,
// with loops a fourth as long, but read the other side's tiles four times as often, and with more LDS each fewer
// run at once.  dk and dv, whose loops go over the heads that share a key head too, gain most.  All gradients in
// us, bf16, without and with shared keys: 4096 tokens of 8 heads of 64 sharing 2, 399 and 145 (124 with shared
// queries as well); 2 x 4096 of 16 sharing 8, 300 and 277; 4 x 4096, 477 and 530.
// With fewer workgroups than the GPU runs at once the tiles of queries are also taken in parts whose sums a further
// launch joins: 4096 tokens of 4 heads of 64 sharing one, 143 us in one part, 82 in four.  Heads of 128 take twice
// the LDS, so that parts serve better than sharing but for few keys and short loops: 4096 tokens of 16 heads
// sharing 4, 391 us with shared keys, 354 in 8 parts (716 in one); 3 x 700 of 6 sharing 3, 67 and 74.  Shared queries
// need fewer workgroups yet where loops are short: the same of 64 channels, 38 us with, 32 without.
struct BwdForm {
    bool share_q, share_k;
    int splits;  // parts that dk and dv are taken in
};
BwdForm bwd_form(const Shape& p, int64_t d, bool is_bf16, int64_t cus) {
    auto workgroups = [&](int64_t tokens, int64_t rows, int64_t heads) {
        const int64_t b = (tokens + rows - 1) / rows;
        return (p.cu_q ? b + p.n - 1 : b * p.n) * heads;
    };
    const int64_t wq = workgroups(p.tq, 32, p.heads), wk = workgroups(p.tk, 32, p.groups);
    const int64_t seen = min((int64_t)p.window + 32, p.tk);  // keys that a block of queries sees
    // tiles of queries that see a block of keys (in packed sequences up to four times as long as their mean)
    const int64_t longest = p.cu_q ? min(p.tq, 4 * p.tq / p.n) : p.tq;
    const int64_t tiles = (min((int64_t)p.window + 32, longest) + 31) / 32 * (p.heads / p.groups);
    BwdForm f{wq <= (d == 64 && seen >= 2048 ? 4 : !is_bf16 || seen >= 1024 ? 2 : 1) * cus,
              d == 64 ? wk <= 8 * cus : wk < (is_bf16 ? cus : cus / 2) && tiles < 128, 1};
    const int64_t least = !is_bf16 ? 4 : f.share_k ? 32 : 16;  // tiles that a part is worth
    const int64_t w = f.share_k ? wk : workgroups(p.tk, 128, p.groups);
    const int64_t want = w == 0 || (d == 64 && !f.share_k) ? 1 : f.share_k ? 2 * cus / w : (3 * cus + w - 1) / w;
    f.splits = (int)max((int64_t)1, min(tiles / least, want));
    return f;
}

template <typename T, int D>
hipError_t run_bwd(const BwdParams& b, const BwdForm& f, hipStream_t stream) {
    constexpr int SW = D * sizeof(T) > 256 ? 2 : 4;  // what LDS has room for
    const hipError_t e = f.share_q ? run_dq<T, D, SW, SW>(b, stream) : run_dq<T, D, 4, 1>(b, stream);
    if (e != hipSuccess) return e;
    return f.share_k ? run_dkv<T, D, SW, SW>(b, f.splits, stream) : run_dkv<T, D, 4, 1>(b, f.splits, stream);
}

}  // namespace attn

namespace {
int64_t stats_bytes(const AttnArgs& a) { return ((a.cu_q ? a.T : a.N * a.T) * a.H * 8 + 15) / 16 * 16; }
}  // namespace

size_t attn_bwd_workspace_bytes(const AttnArgs& a) {
    const int splits = attn::bwd_form(attn_shape(a), a.d, a.dtype_bf16, a.cus).splits;
    return (size_t)(stats_bytes(a) + (splits > 1 ? splits * 2 * (a.cu_q ? a.S : a.N * a.S) * a.G * a.d * 4 : 0));
}

hipError_t launch_attn_bwd(const AttnArgs& a, void* workspace) {
    const int64_t queries = a.cu_q ? a.T : a.N * a.T, keys = a.cu_q ? a.S : a.N * a.S;
    float* stats = static_cast<float*>(workspace);
    const attn::Shape p = attn_shape(a);
    const attn::BwdParams b{(const char*)a.q, (const char*)a.k, (const char*)a.v, (const char*)a.o, (const char*)a.d_o, a.lse,
                            a.dq, a.dk, a.dv, stats, stats + queries * a.H, queries,
                            workspace ? stats + stats_bytes(a) / 4 : nullptr, keys, p};
    const attn::BwdForm f = attn::bwd_form(p, a.d, a.dtype_bf16, a.cus);
    const hipStream_t s = (hipStream_t)a.stream;
    if (a.dtype_bf16) return a.d == 64 ? attn::run_bwd<bf16, 64>(b, f, s) : attn::run_bwd<bf16, 128>(b, f, s);
    return a.d == 64 ? attn::run_bwd<float, 64>(b, f, s) : attn::run_bwd<float, 128>(b, f, s);
}

}  // namespace gdn2
