// gdn2_attn_fwd.hip -- causal attention with shared key heads and an optional window, forward.
//
//   s_ij = scale q_i . k_j for the keys j that query i sees: j <= p_i and j > p_i - window, where
//   query i of lq stands at p_i = lk - lq + i of its sequence's lk keys;
//   o_i = sum_j e^(s_ij - m) v_j / l,  l = sum_j e^(s_ij - m),  lse_i = m + log l.
//
// One pass over the keys with the running maximum m and sum l.  A workgroup of 4 or 8 waves takes 32 queries a wave
// of one head; tiles of keys and values go from memory to LDS directly, one tile ahead of the
// products.  A wave forms S^T = K Q^T, so that a lane holds scores of one query (its column): the
// maximum and the sum are reductions within a lane and with the lane 32 away, and the probabilities
// are the next product's operand (O^T = V^T P^T) as they stand.  S, m, l and O are fp32; with bf16
// inputs a probability is rounded to bf16 once (the matrix unit's operand), the sum l takes it
// unrounded, and o is rounded on the store.
//
// Heads of 128 in bf16, on several cards of one kind: 32768 tokens of one sequence, 16 heads sharing 2, 3.76 to 3.97
// ms (1110 to 1170 TFLOP/s; a product of 16384^3 reaches 1350 to 1380): the matrix units are busy for 52 to 56% of
// the cycles, at a clock that their power brings down to 1.7 to 1.9 GHz.  8 x 4096 tokens, 16 heads sharing 8,
// window 2048, 439 to 470 us (880 to 940 of the scores that are seen): loops of 33 tiles, for which the matrix units
// are busy for 44 to 46% at 1.8 to 1.9 GHz, keys and values are read four times over (1040 MB, 2.3 TB/s) and a
// quarter of the waves' cycles wait.  Two waves a SIMD, 256 registers each.  Heads of 64: 12648 packed tokens of 32
// heads sharing 4, 164 to 171 us (725 to 760), 1040 vector instructions' issue slots (32 exponentials take four each)
// of 1500 cycles a wave and tile of 64 keys; three waves a SIMD (two took 184 us, four spill: 171).  fp32: 2 x 4096
// tokens, 16 heads of 128 sharing 4, 1037 us (133 TFLOP/s; a product of 8192^3 reaches 153); of 64, 587 us (117).
#include "gdn2_attn.h"

namespace gdn2 {
namespace attn {

// keys in a tile
template <typename T, int SW> constexpr int kKeys = sizeof(T) == 2 && SW == 1 ? 64 : 32;
template <typename T, int D, int SW> constexpr int kFwdLds = SW * 2 * 2 * kKeys<T, SW> * Tile<T, D>::kRow;
// Weights are formed against a reference near the row's largest score so far.  The sum over a lane's half of a
// row's part of a tile may grow up to this (in units of the reference's weight) before the reference follows.
constexpr float kSlack = 4096.f;
// So the sums of a row over its tiles, 2^26 at most, are up to 2^39 times a mean of values, and leave fp32 for values
// near its end.  A row that comes to kLarge (or is not finite) is formed again with all its weights scaled by kDamp,
// a power of two that changes no bit of what stays in fp32's range; below kLarge 2^11 waves and parts can be joined.
constexpr float kLarge = 0x1p112f, kDamp = 0x1p-40f;

struct FwdParams {
    const char* q;
    const char* k;
    const char* v;
    void* o;
    float* lse;
    Parts parts;  // of more than one split, or unused
    Shape p;
};

// The work of one workgroup of NW waves.  SW of them share 32 queries: each takes every SWth tile of keys, with
// tiles of its own in LDS, and their sums are joined at the end.  Returns whether some output of a wave is not finite or
// large, and leaves that wave's outputs unwritten (`flag`: in LDS, zero).  A product multiplies what a query does not
// see by zero, which infinities and NaN survive: the form that is not FIRST leaves out value by value what the mask
// hides.  It keeps in `large` (in LDS, zero) whose outputs are not finite or large, of each wave's 32 queries; `damped`,
// it scales their weights, and writes all outputs as they are.
template <typename T, int D, int NW, int SW, bool FIRST>
__device__ __forceinline__ bool fwd_block(const FwdParams& a, Lds base, GDN2_LDS unsigned* flag, GDN2_LDS unsigned* large, bool damped) {
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
    const char* k = a.k + w.s.k0 * p.k_stride + (int64_t)kv * L::kRow;
    const char* v = a.v + w.s.k0 * p.v_stride + (int64_t)kv * L::kRow;
    const int first = w.block * BM, off = lk - lq;  // the block's first query; where query 0 stands

    // the tiles that some query of the block sees
    const int64_t low = (int64_t)off + first, high = off + (int64_t)min(first + BM, lq) - 1;
    const int64_t from = low - p.window + 1;
    int t0 = from > 0 ? (int)(from / BK) : 0;
    const int all = high >= 0 ? (int)(high / BK) + 1 : 0;
    // and those of the workgroup's part of them
    const int per = (max(all - t0, 0) + (int)gridDim.y - 1) / (int)gridDim.y;
    t0 = min(t0 + per * (int)blockIdx.y, all);
    const int t1 = min(t0 + per, all);

    // the wave's queries; a lane's own is column l % 32
    const int mine = first + wave * 32, rows = min(32, lq - mine);
    const int64_t pos0 = (int64_t)off + mine;
    const int pos = (int)(pos0 + (lane & 31));
    const Lds row_base = L::row_base(lane), col_base = L::col_base(lane);
    auto place = [&](int t) { return base + (part * 2 + (t / SW & 1)) * 2 * BYTES; };
    auto stage = [&](int t) {
        const int left = min(BK, lk - t * BK);
        const Lds to = place(t);
        L::template stage<BK, NW / SW>(to, k + (int64_t)t * BK * p.k_stride, span(left, p.k_stride, L::kRow), p.k_stride, wave, lane);
        L::template stage<BK, NW / SW>(to + BYTES, v + (int64_t)t * BK * p.v_stride, span(left, p.v_stride, L::kRow), p.v_stride, wave, lane);
    };
    // the queries come by way of the (first wave's) second tile's place in LDS, if they have room there: rows are read whole
    constexpr bool VIA = BM * L::kRow <= 2 * BYTES;
    const char* qp = a.q + (w.s.q0 + first) * p.q_stride + (int64_t)head * L::kRow;
    Op<T> q[KS];
    if (t0 + part < t1) stage(t0 + part);
    if constexpr (VIA) {
        const Lds to = base + (~(t0 / SW) & 1) * 2 * BYTES;
        L::template stage<BM, NW>(to, qp, span(min(BM, lq - first), p.q_stride, L::kRow), p.q_stride, all_waves, lane);
        tile_barrier();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) q[ks] = L::row_op(row_base + to + wave * 32 * L::kRow, 0, ks);
        if (SW > 1) lds_barrier();
    } else {
        const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(qp), 0, span(min(BM, lq - first), p.q_stride, L::kRow), 0x00020000);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) q[ks] = global_op<T>(r, (wave * 32 + (lane & 31)) * p.q_stride, ks, g);
    }
    f32x16 o[DT];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) o[dt] = zero16();
    float m = -__builtin_inff(), l = 0.f;  // the reference (base 2) and the lane's part of the sum
    const bool damp = !FIRST && damped && (large[wave] >> (lane & 31) & 1);

    f32x16 s[BK / 32];
    auto scores = [&](Lds rb) {
#pragma unroll
        for (int h = 0; h < BK / 32; ++h) {
            s[h] = zero16();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) mma(s[h], L::row_op(rb, 32 * h, ks), q[ks]);
        }
    };
    auto hide = [&](const Seen& seen) {
#pragma unroll
        for (int h = 0; h < BK / 32; ++h)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[h][i] = seen(32 * h + acc_row(i, g)) ? s[h][i] : -__builtin_inff();
    };
    // the largest score becomes the reference, and the sums follow it, for the queries that `need` it
    auto follow = [&](bool need) {
        float top = s[0][0];
#pragma unroll
        for (int h = 0; h < BK / 32; ++h)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[h][i]);
        top = fmaxf(top, other_half(top, lane)) * p.scale_log2;
        const float to = need ? fmaxf(m, top) : m, f = to == m ? 1.f : __builtin_amdgcn_exp2f(m - to);
        m = to;
        l *= f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[dt] *= f;
    };
    // scores become weights; returns their sum
    auto weights = [&] {
        const float ref = m == -__builtin_inff() ? 0.f : m;  // nothing seen yet: all scores are -inf
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < BK / 32; ++h)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[h][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[h][i], p.scale_log2, -ref));
                sum += s[h][i];
            }
        return sum;
    };
    bool first_tile = true;  // of those that the wave has to do with
    for (int t = t0 + part; t < t1; t += SW) {
        if (SW == 1) tile_barrier();
        else own_tile_wait();
        if (t + SW < t1) stage(t + SW);
        const int key0 = t * BK;
        if (rows <= 0 || key0 > pos0 + rows - 1 || key0 + BK - 1 <= pos0 - p.window) continue;  // nothing that the wave's queries see
        const bool cut = key0 + BK - 1 > pos0 || key0 <= pos0 + 31 - p.window;                 // not all that they see
        const Seen seen = seen_between(pos - key0 - p.window + 1, pos - key0);                 // the lane's query's
        const Lds tk = place(t);
        const Lds rb = opaque(row_base + tk);
        scores(rb);
        if (cut) hide(seen);
        if (first_tile) follow(true);
        float sum = weights();
        // The reference is followed only where weights outgrow it (the exponents of fp32 and bf16 have room),
        // or where there is none yet.  Each query goes by its own two halves, and either calls the vote: what a
        // neighbour does changes no bit.
        auto outgrown = [&](float x) { return x > kSlack || (m == -__builtin_inff() && x == x); };
        if (__any(!first_tile && outgrown(sum))) {
            const float other = other_half(sum, lane);  // by all lanes
            const bool need = outgrown(sum) || outgrown(other);
            scores(rb);
            if (cut) hide(seen);
            follow(need);
            sum = weights();
        }
        first_tile = false;
        if (!FIRST) {
            sum *= damp ? kDamp : 1.f;
#pragma unroll
            for (int h = 0; h < BK / 32; ++h)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[h][i] *= damp ? kDamp : 1.f;
        }
        l += sum;
        Op<T> pr[BK / 16];
#pragma unroll
        for (int c = 0; c < BK / 16; ++c) pr[c] = op_of<T>(s[c / 2], c % 2);
        const Lds cb = opaque(col_base + tk + BYTES);
        if (!FIRST && cut) {
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                const f32x16 add = special_sum<T, D, BK>(cb, dt, seen, g, false);
#pragma unroll
                for (int ks = 0; ks < BK / 16; ++ks) mma(o[dt], finite_part<T>(L::col_op(cb, 16 * ks, dt)), pr[ks]);
                o[dt] += add;
            }
            continue;
        }
#pragma unroll
        for (int ks = 0; ks < BK / 16; ++ks)
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) mma(o[dt], L::col_op(cb, 16 * ks, dt), pr[ks]);
    }
    bool any = false;
    if (FIRST || !damped) {
        unsigned top = 0;  // the largest size, as its bits: infinities and NaN are larger
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = max(top, size_bits(o[dt][i]));
        const uint64_t whose = __ballot(top >= size_bits(kLarge));
        const bool again = whose != 0;
        if (again) *flag = 1;
        if (!FIRST && again && lane == 0)
            __hip_atomic_fetch_or(large + wave, (unsigned)whose | (unsigned)(whose >> 32), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        lds_barrier();
        any = *flag != 0;
        if (SW == 1 ? again : any) return any;
    } else {
        lds_barrier();
    }
    if (rows <= 0) return any;
    l += other_half(l, lane);
    const int64_t row0 = (w.s.q0 + mine) * p.heads + head, row = row0 + (int64_t)(lane & 31) * p.heads;
    const bool live = (lane & 31) < rows;
    const int64_t at = (int64_t)blockIdx.y * a.parts.rows + row;
    auto log_sum = [&] { return l == 0.f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(damp ? l / kDamp : l)) * kLn2; };
    auto part_sum = [&] { return float2{m, damp ? -l : l}; };  // the sign says that the part's weights are scaled
    if constexpr (SW > 1) {
        typedef WaveSums<D, SW> Sums;
        static_assert(Sums::kBytes <= kFwdLds<T, D, SW> && SW * 256 <= kFwdLds<T, D, SW>, "room for the sums");
        if (g == 0) *(GDN2_LDS f32x2*)(uintptr_t)(base + (part * 32 + lane) * 8) = f32x2{m, l};
        lds_barrier();
        f32x2 ml[SW];
        float ref = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < SW; ++i) {
            ml[i] = lds_get<f32x2>(base + (i * 32 + (lane & 31)) * 8);
            ref = fmaxf(ref, ml[i][0]);
        }
        l = 0.f;
#pragma unroll
        for (int i = 0; i < SW; ++i) l += ml[i][1] * (ml[i][0] == ref ? 1.f : __builtin_amdgcn_exp2f(ml[i][0] - ref));
        const float f = m == ref ? 1.f : __builtin_amdgcn_exp2f(m - ref);
        m = ref;
        lds_barrier();
        Sums sums;
        sums.add(base, o, f, part, lane);
        if (!live) return any;
        if (gridDim.y > 1) {
            sums.template store<float>(a.parts.o + at * D, 1.f, part, g);
            if (g == 0 && part == 0) a.parts.ml[at] = part_sum();
            return any;
        }
        sums.template store<T>((T*)a.o + row * D, l == 0.f ? 0.f : 1.f / l, part, g);
        if (a.lse && g == 0 && part == 0) a.lse[row] = log_sum();
        return any;
    }
    if (gridDim.y > 1) {
        if (live) {
            store_column<float, D>(a.parts.o + at * D, o, 1.f, g);
            if (g == 0) a.parts.ml[at] = part_sum();
        }
        return any;
    }
    if (a.lse && live && g == 0) a.lse[row] = log_sum();
    store_rows<T, D>(base + wave * 32 * L::kRow, (char*)a.o + row0 * L::kRow, (int64_t)p.heads * L::kRow, rows, o, l == 0.f ? 0.f : 1.f / l, lane);
    return any;
}
// a call of its own, so that the kernel keeps its registers to the first form; `outcome`: a flag, and `large`
template <typename T, int D, int NW, int SW>
__device__ __attribute__((noinline)) void fwd_again(FwdParams a, Lds base, GDN2_LDS unsigned* outcome) {
    if (threadIdx.x < NW / SW) outcome[1 + threadIdx.x] = 0;
#pragma unroll 1
    for (int damped = 0; damped < 2; ++damped) {
        if (threadIdx.x == 0) *outcome = 0;
        __syncthreads();
        if (!fwd_block<T, D, NW, SW, false>(a, base, outcome, outcome + 1, damped != 0)) break;
        __syncthreads();
    }
}

template <typename T, int D, int NW, int SW>
__global__ __launch_bounds__(NW * 64, SW > 1 ? (kFwdLds<T, D, SW> > 80000 ? 1 : 2) : D == 64 ? 3 : 2) void fwd_kernel(FwdParams a) {
    __shared__ __attribute__((aligned(1024))) char lds[kFwdLds<T, D, SW>];
    __shared__ unsigned words[1 + NW / SW];
    GDN2_LDS unsigned* outcome = (GDN2_LDS unsigned*)words;
    if (threadIdx.x == 0) *outcome = 0;
    if (fwd_block<T, D, NW, SW, true>(a, lds_of(lds), outcome, nullptr, false)) {
        __syncthreads();
        fwd_again<T, D, NW, SW>(a, lds_of(lds), outcome);
    }
}

// Joins parts: a workgroup a row, D / 4 threads a part; each takes every SUBth part, several loads at once.
template <typename T, int D>
__global__ __launch_bounds__(256) void join_kernel(Parts p, T* __restrict__ o, float* __restrict__ lse, Owned owned) {
    constexpr int SUB = 256 / (D / 4);
    __shared__ f32x4 sum[SUB][D / 4];
    __shared__ float total[SUB];
    const int64_t row = blockIdx.x;
    const int c = threadIdx.x % (D / 4), sub = threadIdx.x / (D / 4), lane = threadIdx.x & 63;
    if (owned.cu) {  // a token of no sequence has no parts and stays as it was
        const int64_t token = row / owned.heads;
        bool found = false;
        for (int64_t base = 0; base < owned.n && !found; base += 64) {
            bool here = false;
            if (base + lane < owned.n) {
                const int64_t lo = clamp64(owned.cu[base + lane], 0, owned.total);
                here = lo <= token && token < clamp64(owned.cu[base + lane + 1], lo, owned.total);
            }
            found = __any(here);
        }
        if (!found) return;
    }
    float m = -__builtin_inff();
    bool damped = false;  // some part's weights are scaled: the other parts' are, too
    for (int i = lane; i < p.splits; i += 64) {
        const float2 ml = p.ml[i * p.rows + row];
        m = fmaxf(m, ml.x);
        damped = damped || ml.y < 0.f;
    }
#pragma unroll
    for (int s = 32; s >= 1; s /= 2) m = fmaxf(m, __shfl_xor(m, s));
    damped = __any(damped);
    f32x4 x{0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
#pragma unroll 4
    for (int i = sub; i < p.splits; i += SUB) {
        const float2 ml = p.ml[i * p.rows + row];
        const f32x4 v = *reinterpret_cast<const f32x4*>(p.o + (i * p.rows + row) * D + 4 * c);
        // a part that saw nothing is all zeros
        const float f = (ml.x == -__builtin_inff() && ml.y == 0.f ? 0.f : __builtin_amdgcn_exp2f(ml.x - m)) *
                        (damped && !(ml.y < 0.f) ? kDamp : 1.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += f * v[e];
        l += f * fabsf(ml.y);
    }
    sum[sub][c] = x;
    if (c == 0) total[sub] = l;
    __syncthreads();
    if (sub == 0) {
#pragma unroll
        for (int s = 1; s < SUB; ++s) {
            x += sum[s][c];
            l += total[s];
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float out[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
        store_vec_any<T, 4>(o + row * D + 4 * c, out);
        if (lse && c == 0) lse[row] = l == 0.f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(damped ? l / kDamp : l)) * kLn2;
    }
}

hipError_t launch_join(const Parts& p, void* o, float* lse, int64_t d, bool bf16_out, const Owned& owned, hipStream_t stream) {
    const dim3 grid((unsigned)p.rows), block(256);
    if (bf16_out && d == 64) hipLaunchKernelGGL((join_kernel<bf16, 64>), grid, block, 0, stream, p, (bf16*)o, lse, owned);
    else if (bf16_out) hipLaunchKernelGGL((join_kernel<bf16, 128>), grid, block, 0, stream, p, (bf16*)o, lse, owned);
    else if (d == 64) hipLaunchKernelGGL((join_kernel<float, 64>), grid, block, 0, stream, p, (float*)o, lse, owned);
    else hipLaunchKernelGGL((join_kernel<float, 128>), grid, block, 0, stream, p, (float*)o, lse, owned);
    return hipGetLastError();
}

// How the forward pass is launched.  Workgroups whose waves share 32 queries are four times as many, and their
// loops a fourth as long, but they read keys and values four times as often: they are taken while they fit the
// GPU in about two rounds (fp32 heads of 128, which two waves share: while they leave most of it idle).  bf16 in
// us, without and with: 4096 tokens of 4 heads of 64 sharing one, 39 and 24; of 8 sharing 2, 59 and 35; of 16
// sharing 4, 60 and 63; heads of 128: 1024 tokens of 4 heads, 24 and 15; of 16, 25 and 22; 4096 of 8, 83 and 96.
// With few workgroups and many keys a block's keys are also taken in parts, as many as fill the GPU, whose sums
// a second launch joins: 4096 tokens of one head of 64 take 18 us in 4 parts, 23 in one.  (Sequences that
// are packed may be shorter than the longest: their parts are, too.)
// Many long sequences without a window take heads of 128 in bf16 256 queries a workgroup, which reads keys and
// values half as often: 32768 tokens of 16 heads, 3948 us at 128, 3827 at 256; 2 x 4096 of 16, 150 and 134.  With
// a window the wider block sees more tiles than its waves use (8 x 4096, window 2048: 434 and 441), and short
// sequences fill it badly (16 x 700: 51 and 58).
struct FwdForm {
    bool share;
    int splits;
    bool wide;
};
FwdForm fwd_form(Shape p, int64_t d, bool is_bf16, int64_t cus) {
    if (deal(&p, p.tq, 128, p.heads / p.groups) <= 0) return {false, 1, false};
    auto workgroups = [&](int64_t rows) {
        const int64_t b = (p.tq + rows - 1) / rows;
        return (p.cu_q ? b + p.n - 1 : b * p.n) * p.heads;
    };
    const bool share = workgroups(32) <= (d == 64 ? 4 * cus : is_bf16 ? 2 * cus : cus / 4);
    const int64_t w = workgroups(share ? 32 : 128), keys = min((int64_t)p.window + (share ? 32 : 128), p.tk);
    const int64_t least = is_bf16 ? 1024 : 256;  // keys of a part: below, the second launch costs more
    bool wide = is_bf16 && d == 128 && !p.cu_q && p.window >= p.tk && p.tq >= 2048 && workgroups(256) >= 2 * cus;
    if (wide) wide = deal(&p, p.tq, 256, p.heads / p.groups) < kMaxGrid / 2;  // of 512 threads
    return {share, w >= cus ? 1 : (int)max((int64_t)1, min(keys / least, 2 * cus / w)), wide};
}

template <typename T, int D, int NW, int SW>
hipError_t run_fwd(FwdParams f, hipStream_t stream) {
    const int64_t grid = deal(&f.p, f.p.tq, NW / SW * 32, f.p.heads / f.p.groups);
    if (grid < 0) return hipErrorInvalidValue;
    if (grid == 0) return hipSuccess;
    hipLaunchKernelGGL((fwd_kernel<T, D, NW, SW>), dim3((unsigned)grid, (unsigned)f.parts.splits), dim3(NW * 64), 0, stream, f);
    if (f.parts.splits > 1)
        return launch_join(f.parts, f.o, f.lse, D, sizeof(T) == 2, Owned{f.p.cu_q, f.p.n, f.p.tq, f.p.heads}, stream);
    return hipGetLastError();
}
template <typename T, int D>
hipError_t choose_fwd(const FwdParams& f, const FwdForm& form, hipStream_t stream) {
    constexpr int SW = D * sizeof(T) > 256 ? 2 : 4;
    if (form.share) return run_fwd<T, D, SW, SW>(f, stream);
    if constexpr (sizeof(T) == 2 && D == 128) {
        if (form.wide) return run_fwd<T, D, 8, 1>(f, stream);
    }
    return run_fwd<T, D, 4, 1>(f, stream);
}

}  // namespace attn

// a window that no sequence is longer than, so that a position less it stays a 32-bit number
constexpr int kAllKeys = INT32_MAX - 1024;

attn::Shape attn_shape(const AttnArgs& a) {
    attn::Shape p{};
    const uint32_t es = a.dtype_bf16 ? 2 : 4;
    p.cu_q = a.cu_q;
    p.cu_k = a.cu_k;
    p.n = a.N;
    p.tq = a.T;
    p.tk = a.S;
    p.heads = (int)a.H;
    p.groups = (int)a.G;
    p.window = a.window > 0 && a.window < kAllKeys ? (int)a.window : kAllKeys;
    p.q_stride = (uint32_t)a.q_stride * es;
    p.k_stride = (uint32_t)a.k_stride * es;
    p.v_stride = (uint32_t)a.v_stride * es;
    p.scale = a.scale;
    p.scale_log2 = a.scale * attn::kLog2e;
    return p;
}

// the launches with the most workgroups: of 128 queries a head, and of 128 keys a key head
bool attn_grid_ok(const AttnArgs& a) {
    attn::Shape p = attn_shape(a);
    const int64_t tokens = a.cu_q ? a.T : a.N * a.T;
    return attn::deal(&p, a.T, 128, p.heads / p.groups) >= 0 && attn::deal(&p, a.S, 128, 1) >= 0 && tokens < ((int64_t)1 << 29);
}

size_t attn_fwd_workspace_bytes(const AttnArgs& a) {
    const int splits = attn::fwd_form(attn_shape(a), a.d, a.dtype_bf16, a.cus).splits;
    return splits > 1 ? attn::parts_bytes((a.cu_q ? a.T : a.N * a.T) * a.H, a.d, splits) : 0;
}

hipError_t launch_attn_fwd(const AttnArgs& a, void* workspace) {
    const attn::Shape p = attn_shape(a);
    const int64_t rows = (a.cu_q ? a.T : a.N * a.T) * a.H;
    const attn::FwdForm form = attn::fwd_form(p, a.d, a.dtype_bf16, a.cus);
    const attn::FwdParams f{(const char*)a.q, (const char*)a.k, (const char*)a.v, a.o, a.lse,
                            attn::parts_in(workspace, rows, a.d, workspace ? form.splits : 1), p};
    const hipStream_t s = (hipStream_t)a.stream;
    if (a.dtype_bf16) return a.d == 64 ? attn::choose_fwd<bf16, 64>(f, form, s) : attn::choose_fwd<bf16, 128>(f, form, s);
    return a.d == 64 ? attn::choose_fwd<float, 64>(f, form, s) : attn::choose_fwd<float, 128>(f, form, s);
}

}  // namespace gdn2
