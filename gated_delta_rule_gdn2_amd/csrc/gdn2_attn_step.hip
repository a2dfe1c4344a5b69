// gdn2_attn_step.hip -- attention of one token for each of N sequences over caches that keep the last
// C tokens: token p lies in slot p mod C.
//
//   o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),  s_j = scale q . k_j,  over the last
//   min(p + 1, window, C) tokens, the sequence's token p (whose key and value the call brings) among
//   them.  The call writes them into slot p mod C; a position below 0 is no token: its output is zero
//   and its cache is left alone.
//
// Bound by reading the caches once.  The query heads of a key head (up to 32 a workgroup) are the
// columns of one product, so that a key is read once for all of them.  A workgroup takes a part of the
// tokens; its waves take tiles of 32 of them in turn, each through LDS of its own and ahead of their use,
// so no barrier stops the loads.  Every wave keeps a maximum, a sum and an output of its own; they are
// joined at the end, and parts of a sequence in a second launch.
//
// 256 sequences over 2048 tokens, 16 heads of 128 sharing 2, bf16: 79 us, 5.0 TB/s (a copy of 2 GiB: 4.9).  3
// sequences over 16384: 16 to 17 us and 4 for the join, of which 10 are the bytes at that rate: 384 workgroups, of
// which a CU has room for one, so that half of them wait for the first.
#include "gdn2_attn.h"

namespace gdn2 {
namespace attn {

struct StepParams {
    const char* q;
    const char* k;
    const char* v;
    char* k_cache;
    char* v_cache;
    const int64_t* positions;
    void* o;
    Parts parts;
    int64_t n, cache, window;
    uint32_t heads, groups;
    int64_t q_stride, k_stride, v_stride;  // bytes between tokens
    float scale_log2;
};

constexpr int kStepKeys = 32;
constexpr int kStepWaves = 4;

__device__ __forceinline__ void arrived(Op<bf16>& x) { asm volatile("" : "+v"(x.v)); }
__device__ __forceinline__ void arrived(Op<float>& x) {
#pragma unroll
    for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(x.v[e]));
}

// all but a wave's last LEFT loads have arrived
template <int LEFT> __device__ __forceinline__ void arrive() {
    __builtin_amdgcn_s_waitcnt(0x0f70 | (LEFT & 15) | (LEFT >> 4) << 14);
    asm volatile("" ::: "memory");
}
// a wave has read what it asked LDS for, and what it wrote there can be read
__device__ __forceinline__ void have_read() {
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
}

template <typename T, int D>
__global__ __launch_bounds__(64 * kStepWaves, 1) void step_kernel(StepParams a) {
    typedef Tile<T, D> L;
    constexpr int NW = kStepWaves, KS = D / 16, DT = D / 32, BYTES = kStepKeys * L::kRow, LOADS = BYTES / 1024;
    constexpr int ROW = D + 4;  // floats of a row of the join: rows 4 banks apart
    // In bf16 the next tile's keys and values are on their way while a tile is used.  In fp32, whose tiles are twice
    // the bytes, the next keys' place is the keys', and they come while weights and values are multiplied; values
    // come while scores are formed: either takes the matrix units longer than a load.  So four waves have room for
    // heads of 128 (64 sequences over 4096 tokens, 16 heads sharing 2: 122 us; 189 with two waves, tiles ahead).
    constexpr bool TWO = sizeof(T) == 2;
    constexpr int TILES = NW * (TWO ? 4 : 2) * BYTES, JOIN = NW * 32 * ROW * 4;
    __shared__ __attribute__((aligned(1024))) char lds[TILES > JOIN ? TILES : JOIN];
    __shared__ float2 ml[NW][32];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t share = a.heads / a.groups, blocks = (share + 31) / 32;
    const uint32_t part = blockIdx.x % a.parts.splits, rest = blockIdx.x / a.parts.splits;
    const uint32_t hb = rest % blocks, kv = rest / blocks % a.groups;
    const int64_t n = rest / blocks / a.groups;
    const int heads = min((int)share - (int)hb * 32, 32);     // of the workgroup
    const int64_t head0 = (int64_t)kv * share + hb * 32;      // the first of them
    const int64_t pos = a.positions[n];
    const int64_t seen = pos < 0 ? 0 : min(pos, min(a.window, a.cache) - 1) + 1;  // tokens, the newest last
    const int64_t newest = seen > 0 ? pos % a.cache : 0;      // its slot
    int64_t oldest = newest - seen + 1;
    if (oldest < 0) oldest += a.cache;
    const int64_t tiles = (seen + kStepKeys - 1) / kStepKeys, per = (tiles + a.parts.splits - 1) / a.parts.splits;
    const int64_t t0 = min(per * part, tiles), t1 = min(t0 + per, tiles);

    const int64_t row_bytes = (int64_t)a.groups * L::kRow, head_off = (int64_t)kv * L::kRow;
    const char* kin = a.k + n * a.k_stride + head_off;
    const char* vin = a.v + n * a.v_stride + head_off;
    char* kc = a.k_cache + n * a.cache * row_bytes + head_off;
    char* vc = a.v_cache + n * a.cache * row_bytes + head_off;
    if (seen > 0 && t1 == tiles && t0 < t1 && hb == 0) {  // the part that holds the newest token keeps it
        const int u = tid;
        if (u < L::kUnits)
            *reinterpret_cast<u32x4*>(kc + newest * row_bytes + u * 16) = *reinterpret_cast<const u32x4*>(kin + u * 16);
        else if (u < 2 * L::kUnits)
            *reinterpret_cast<u32x4*>(vc + newest * row_bytes + (u - L::kUnits) * 16) =
                *reinterpret_cast<const u32x4*>(vin + (u - L::kUnits) * 16);
    }

    f32x16 o[DT];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) o[dt] = zero16();
    float m = -__builtin_inff(), l = 0.f;

    const Lds mine = lds_of(lds) + wave * (TWO ? 4 : 2) * BYTES, row_base = L::row_base(lane), col_base = L::col_base(lane);
    // Tile t's keys and values.  The newest token comes from the call: its slot is being written.  Rows
    // behind it repeat it, until their values become zeros: weights of zero would make NaN of its infinities.
    auto stage = [&](int64_t t, int buf, bool keys, bool values) {
        const Lds at = mine + buf * 2 * BYTES;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int u = i * 64 + lane, row = u / L::kUnits, off = ((u % L::kUnits) ^ L::swz(row)) << 4;
            const int64_t token = t * kStepKeys + row;
            int64_t slot = oldest + token;
            if (slot >= a.cache) slot -= a.cache;
            const bool last = token >= seen - 1;
            if (keys) load_far_to_lds(at + i * 1024, (last ? kin : kc + slot * row_bytes) + off);
            if (values) load_far_to_lds(at + BYTES + i * 1024, (last ? vin : vc + slot * row_bytes) + off);
        }
    };
    int buf = 0;
    if (t0 + wave < t1) stage(t0 + wave, 0, true, true);
    Op<T> q[KS];
    {
        const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(a.q + n * a.q_stride + head0 * L::kRow), 0, heads * L::kRow, 0x00020000);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) q[ks] = global_op<T>(r, (lane & 31) * L::kRow, ks, g);
    }
    // waited for here, or the compiler waits for every load in flight in each turn of the loop
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) arrived(q[ks]);
    for (int64_t t = t0 + wave; t < t1; t += NW) {
        const bool more = t + NW < t1;
        if (TWO && more) stage(t + NW, buf ^ 1, true, true);
        if (TWO && more) arrive<2 * LOADS>();  // this tile's
        else if (TWO) arrive<0>();
        else arrive<LOADS>();                  // this tile's keys
        const Lds tk = mine + buf * 2 * BYTES;
        const Lds rb = opaque(row_base + tk), cb = opaque(col_base + tk + BYTES);
        f32x16 s = zero16();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) mma(s, L::row_op(rb, 0, ks), q[ks]);
        if (!TWO) have_read();
        if (!TWO && more) stage(t + NW, 0, true, false);
        const int64_t left = seen - t * kStepKeys;
        if (left < kStepKeys) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = acc_row(i, g) < (int)left ? s[i] : -__builtin_inff();
        }
        float top = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
        top = fmaxf(top, other_half(top, lane)) * a.scale_log2;
        if (__any(top > m)) {
            const float next = fmaxf(m, top), f = next == m ? 1.f : __builtin_amdgcn_exp2f(m - next);
            m = next;
            l *= f;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) o[dt] *= f;
        }
        const float ref = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], a.scale_log2, -ref));
            l += s[i];
        }
        const Op<T> pr[2] = {op_of<T>(s, 0), op_of<T>(s, 1)};
        if (!TWO && more) arrive<LOADS>();  // its values
        else if (!TWO) arrive<0>();
        if (left < kStepKeys) {  // the wave's last tile, all of which is there
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                if ((i * 64 + lane) / L::kUnits >= (int)left)
                    *(GDN2_LDS u32x4*)(uintptr_t)(tk + BYTES + (i * 64 + lane) * 16) = u32x4{0, 0, 0, 0};
            have_read();
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) mma(o[dt], L::col_op(cb, 16 * ks, dt), pr[ks]);
        have_read();  // before the next loads into the place are given out
        if (!TWO && more) stage(t + NW, 0, false, true);
        if (TWO) buf ^= 1;
    }
    l += other_half(l, lane);

    // the waves' parts
    __syncthreads();
    const int col = lane & 31;
    float* join = reinterpret_cast<float*>(lds);
    if (col < heads) {
        store_column<float, D>(join + (wave * 32 + col) * ROW, o, 1.f, g);
        if (g == 0) ml[wave][col] = float2{m, l};
    }
    __syncthreads();
    const int64_t row0 = n * a.heads + head0;
    for (int i = tid; i < heads * (D / 4); i += 64 * NW) {
        const int h = i / (D / 4), c = i % (D / 4) * 4;
        float top = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, ml[w][h].x);
        float sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float2 y = ml[w][h];
            const float f = y.x == -__builtin_inff() ? (y.y == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(y.x - top);
            sum += f * y.y;
            const f32x4 v = *reinterpret_cast<const f32x4*>(join + (w * 32 + h) * ROW + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] += f * v[e];
        }
        if (a.parts.splits > 1) {
            const int64_t at = (int64_t)part * a.parts.rows + row0 + h;
            store_vec_any<float, 4>(a.parts.o + at * D + c, x);
            if (c == 0) a.parts.ml[at] = float2{top, sum};
        } else {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] *= inv;
            store_vec_any<T, 4>(reinterpret_cast<T*>(a.o) + (row0 + h) * D + c, x);
        }
    }
}

// Parts of a sequence: up to two workgroups a CU, of whole turns of the waves, and no more of them than those turns
// need.  (LDS has room for two at once at 64 channels and for one at 128.)
int step_splits(const AttnStepArgs& a) {
    const int64_t share = a.H / a.G, groups = a.N * a.G * ((share + 31) / 32);
    const int waves = kStepWaves;
    const int64_t seen = a.window > 0 && a.window < a.C ? a.window : a.C, turns = (seen + kStepKeys * waves - 1) / (kStepKeys * waves);
    const int64_t want = max((int64_t)1, 2 * (int64_t)a.cus / groups), each = (turns + want - 1) / want;
    return (int)((turns + each - 1) / each);
}

template <typename T, int D>
hipError_t run_step(const StepParams& p, hipStream_t stream) {
    const int64_t share = p.heads / p.groups, grid = p.n * p.groups * ((share + 31) / 32) * p.parts.splits;
    hipLaunchKernelGGL((step_kernel<T, D>), dim3((unsigned)grid), dim3(64 * kStepWaves), 0, stream, p);
    if (p.parts.splits > 1) return launch_join(p.parts, p.o, nullptr, D, sizeof(T) == 2, Owned{}, stream);
    return hipGetLastError();
}

}  // namespace attn

size_t attn_step_workspace_bytes(const AttnStepArgs& a) {
    const int splits = attn::step_splits(a);
    return splits > 1 ? attn::parts_bytes(a.N * a.H, a.d, splits) : 0;
}

hipError_t launch_attn_step(const AttnStepArgs& a, void* workspace) {
    const int64_t es = a.dtype_bf16 ? 2 : 4;
    attn::StepParams p{(const char*)a.q, (const char*)a.k, (const char*)a.v, (char*)a.k_cache, (char*)a.v_cache, a.positions, a.o,
                       attn::parts_in(workspace, a.N * a.H, a.d, workspace ? attn::step_splits(a) : 1), a.N, a.C,
                       a.window > 0 ? a.window : a.C, (uint32_t)a.H, (uint32_t)a.G, a.q_stride * es, a.k_stride * es, a.v_stride * es,
                       a.scale * attn::kLog2e};
    const hipStream_t s = (hipStream_t)a.stream;
    if (a.dtype_bf16) return a.d == 64 ? attn::run_step<bf16, 64>(p, s) : attn::run_step<bf16, 128>(p, s);
    return a.d == 64 ? attn::run_step<float, 64>(p, s) : attn::run_step<float, 128>(p, s);
}

}  // namespace gdn2
