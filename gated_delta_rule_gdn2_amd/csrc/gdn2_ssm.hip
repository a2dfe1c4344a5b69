// gdn2_ssm.hip -- the selective state space scan over prompts, and its step for single tokens.
//
// Per sequence and head, with a state S of dk rows and dv columns:
//   dt_t = softplus(raw_t + bias),  S_t = exp(dt_t A) S_{t-1} + dt_t b_t x_t^T,
//   y_t = S_t^T c_t + D x_t
// b and c belong to a group of heads; the columns of S are independent.
//
// In a chunk of 64 tokens with the state S that enters it and cum_i = sum_{s<=i} dt_s A:
//   M[i,j] = (c_i . b_j) exp(cum_i - cum_j) dt_j   (j <= i, else 0)
//   y_i    = exp(cum_i) S^T c_i + sum_j M[i,j] x_j + D x_i
//   S'     = exp(cum_63) S + sum_j b_j (exp(cum_63 - cum_j) dt_j x_j)^T
// All four products run on the matrix units.
#include "gdn2_bf16_ops.h"
#include "gdn2_device.h"
#include "gdn2_launch.h"

namespace gdn2 {
namespace ssm {

constexpr int Q = 64;  // tokens of a chunk

constexpr int AHEAD = 4;  // chunks whose decays are formed together

typedef uint32_t U4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// raw + bias, through softplus where asked: max(v, 0) + log(1 + e^-|v|).  The library's log1p and
// exp: once per token and head, and final states keep their fp32 accuracy.
__device__ __forceinline__ float time_step(float v, bool softplus) {
    return softplus ? fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))) : v;
}

// v of another lane by a DPP control, 0 where there is none (rows: the 16-lane rows that take it)
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (uint32_t)u, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// inclusive sums over the wave's lanes: shifts within rows of 16, then each row's sum to the rows
// behind it.  In LDS permutes the same sums kept a wave, and the barrier it reaches last, 3000
// cycles a chunk.
__device__ __forceinline__ double scan(double v) {
    v += dpp<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
    v += dpp<0x112, 0xf>(v);
    v += dpp<0x114, 0xf>(v);
    v += dpp<0x118, 0xf>(v);
    v += dpp<0x142, 0xa>(v);  // row_bcast 15 to rows 1 and 3
    v += dpp<0x143, 0xc>(v);  // row_bcast 31 to rows 2 and 3
    return v;
}
__device__ __forceinline__ double last_lane(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, 63), hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// e^v, rounded to fp32 once before the hardware's base-2 exponential
__device__ __forceinline__ float exp_of(double v) { return __builtin_amdgcn_exp2f((float)(v * 1.4426950408889634)); }

__device__ __forceinline__ bool is_finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }

// ---- LDS tiles ------------------------------------------------------------------------------
// [64 tokens][W] row-major, in 16-byte units whose place in the row is XORed with a function of
// the row.  Measured phases of the 64 banks: a 16-byte read takes lanes 0-3, 12-15 and 20-27
// together (then their like), 8-byte and 4-byte reads 32 lanes in a row.  So a 16-byte read of 16
// rows (kRows: products over W) wants the rows of a phase at different units, the transposing
// 8-byte read (kCols: products over tokens; 8 rows, two units of each) different pairs of units
// over 8 rows.  b is read both ways, c only by rows, x by columns and 8 bytes of 16 rows (kBoth).
// Without the difference between them a sixth of the chunk kernel's time was LDS conflicts.
enum Reads { kRows, kCols, kBoth };
template <typename T, int W, Reads R>
struct Tile {
    static constexpr int UPR = W * (int)sizeof(T) / 16;  // units per row
    static constexpr int EPU = 16 / (int)sizeof(T);      // elements per unit
    __device__ static __forceinline__ int swz(int row) {
        const int r = UPR >= 16 ? row : row >> 1;  // an 8-unit row is half of the banks
        if constexpr (R == kRows || sizeof(T) == 4) return r & (UPR >= 16 ? 15 : 7);
        else if constexpr (UPR >= 16) return ((r & 7) << 1) | (R == kBoth ? (r >> 3) & 1 : 0);
        else return ((r & 3) << 1) | (R == kBoth ? (r >> 2) & 1 : 0);
    }
    static constexpr int RB = UPR * 16;  // bytes of a row
    // Byte offset of (row, col).  A row of 16 R + row adds 16 R rows; a column whose bits above a
    // lane's own are c enters by XOR with its bytes: a pattern's every address is one lane base,
    // XORed with one constant and offset by another.
    __device__ static __forceinline__ int at(int row, int col) {
        return row * RB + ((col * (int)sizeof(T)) ^ (swz(row) << 4));
    }
};

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> lds_vec(const void* tile, int off) {
    return load_vec<T, N>(reinterpret_cast<const T*>(static_cast<const char*>(tile) + off));
}

// Operands.  `base` is the pattern's lane base: rows_base, perm_base or cols_base.
// A product over W: row r0 + lane % 16, elements col + 8g .. col + 8g + 7.
template <typename TL>
__device__ __forceinline__ int rows_base(int lane) { return TL::at(lane & 15, (lane >> 4) * 8); }
template <typename TL>
__device__ __forceinline__ Frag<bf16> rows_contig(const bf16* t, int base, int r0, int col) {
    Frag<bf16> f;
    const Vec<bf16, 8> v = lds_vec<bf16, 8>(t, (base ^ (col * 2)) + r0 * TL::RB);
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = v.v[e];
    return f;
}
template <typename TL>
__device__ __forceinline__ Frag<float> rows_contig(const float* t, int base, int r0, int col) {
    Frag<float> f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const Vec<float, 4> v = lds_vec<float, 4>(t, (base ^ ((col + 4 * h) * 4)) + r0 * TL::RB);
#pragma unroll
        for (int e = 0; e < 4; ++e) f.v[4 * h + e] = v.v[e];
    }
    return f;
}
// The same in the permuted map: elements col + 4g .. + 3 and col + 16 + 4g .. + 3.  The rows too
// enter by XOR (16 rows are a power of two of bytes): two 8-byte reads that differ by a constant the
// compiler merges into one, which runs in the phases of a 16-byte read with both of a lane's
// halves in the same banks.
template <typename TL>
__device__ __forceinline__ int perm_base(int lane) { return TL::at(lane & 15, (lane >> 4) * 4); }
template <typename TL, typename T>
__device__ __forceinline__ Frag<T> rows_perm(const T* t, int base, int r0, int col) {
    Frag<T> f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const Vec<T, 4> v = lds_vec<T, 4>(t, base ^ ((col + 16 * h) * (int)sizeof(T) + r0 * TL::RB));
#pragma unroll
        for (int e = 0; e < 4; ++e) f.v[4 * h + e] = v.v[e];
    }
    return f;
}
// A product over tokens, in the permuted map: column col + lane % 16, tokens t0 + 4g + e and
// t0 + 16 + 4g + e.  bf16 through the transposing LDS read: the 16 lanes of a group read four rows
// of 16 columns, 8 bytes each, and get a column each.
template <typename TL, typename T>
__device__ __forceinline__ int cols_base(int lane) {
    if constexpr (sizeof(T) == 2) return TL::at((lane >> 4) * 4 + ((lane >> 2) & 3), (lane & 3) * 4);
    else return TL::at((lane >> 4) * 4, lane & 15);
}
template <typename TL>
__device__ __forceinline__ Frag<bf16> cols_perm(const bf16* t, int base, int t0, int col) {
    typedef __attribute__((address_space(3))) s16x4* Lds;
    Frag<bf16> f;
    const char* p = reinterpret_cast<const char*>(t) + (base ^ (col * 2)) + t0 * TL::RB;
    const bf16x4 lo = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)p));
    const bf16x4 hi = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p + 16 * TL::RB)));
    f.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return f;
}
template <typename TL>
__device__ __forceinline__ Frag<float> cols_perm(const float* t, int base, int t0, int col) {
    Frag<float> f;
#pragma unroll
    for (int e = 0; e < 8; ++e)  // a row of 4g + e: e is in the swizzle's low bits
        f.v[e] = lds_vec<float, 1>(t, (base ^ (col * 4) ^ ((e & 3) << 4)) + (t0 + (e >> 2) * 16 + (e & 3)) * TL::RB).v[0];
    return f;
}

// A lane's base that the compiler may not keep derived addresses of: they are one XOR each, and all
// of them in registers were spilled.
__device__ __forceinline__ int fresh(int base) {
    asm volatile("" : "+v"(base));
    return base;
}

// ---- weighted x -----------------------------------------------------------------------------
// The state is fp32 and is returned, so its update keeps 24 bits: in bf16 x and b are exact and
// the product weight * x is carried as three bf16 planes; in fp32 it is one.
template <typename T> struct Planes;
template <> struct Planes<bf16> {
    static constexpr int N = 3;
    Frag<bf16> p[3];
    // elements e and e + 1, e even: one conversion packs two
    __device__ __forceinline__ void set(const Frag<bf16>& x, int e, float w0, float w1) {
        f32x2 v = {(float)x.v[e] * w0, (float)x.v[e + 1] * w1};
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const bf16x2 r = __builtin_convertvector(v, bf16x2);
            p[i].v[e] = r[0];
            p[i].v[e + 1] = r[1];
            const uint32_t u = __builtin_bit_cast(uint32_t, r);
            v[0] -= __uint_as_float(u << 16);
            v[1] -= __uint_as_float(u & 0xffff0000u);
        }
    }
    // the compiler may not move the forming behind this
    __device__ __forceinline__ void formed() {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            U4 u = __builtin_bit_cast(U4, p[i].v);
            asm volatile("" : "+v"(u));
            p[i].v = __builtin_bit_cast(bf16x8, u);
        }
    }
};
template <> struct Planes<float> {
    static constexpr int N = 1;
    Frag<float> p[1];
    __device__ __forceinline__ void set(const Frag<float>& x, int e, float w0, float w1) {
        p[0].v[e] = x.v[e] * w0;
        p[0].v[e + 1] = x.v[e + 1] * w1;
    }
    __device__ __forceinline__ void formed() {
#pragma unroll
        for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(p[0].v[e]));
    }
};

// A token's logarithm of decay, no less than 160 factors of two: an fp32 decay is 0 from 150 on, so
// no result differs, and a token that clears the state leaves the sums of those behind it exact
// enough.  (At -1e7 the difference of two such sums in fp32 was off by e; -inf gave NaN.)  NaN stays.
__device__ __forceinline__ double log_decay(float dt, float A) {
    constexpr double least = -110.9035488896;  // 160 ln 2
    const double v = (double)dt * (double)A;
    return v < least ? least : v;
}

// Sums of logarithms of decays are formed in 64 bits.  What a pair of tokens needs, the decay
// between them, is a difference of two: in bf16 of their fp32 roundings (to base 2, for the
// hardware's exponential; an error of |cum| 2^-23, far below a bf16 rounding of M where M counts),
// in fp32 of the 64-bit sums.
template <typename T> struct Pair {
    typedef float Cum;
    __device__ static __forceinline__ Cum cum(double v) { return (float)(v * 1.4426950408889634); }
    __device__ static __forceinline__ float decay(Cum i, Cum j) { return __builtin_amdgcn_exp2f(i - j); }
    __device__ static __forceinline__ float decay(Cum i) { return __builtin_amdgcn_exp2f(i); }
};
template <> struct Pair<float> {
    typedef double Cum;
    __device__ static __forceinline__ Cum cum(double v) { return v; }
    __device__ static __forceinline__ float decay(Cum i, Cum j) { return exp_of(i - j); }
    __device__ static __forceinline__ float decay(Cum i) { return exp_of(i); }
};

struct Params {
    const void* x;
    const void* dt;
    const void* b;
    const void* c;
    const float* A;
    const float* D;
    const float* dt_bias;
    const float* s0;
    void* y;
    float* sT;
    const int64_t* cu;
    int64_t T;
    int N, H, G, dv;
    int xs, dts, bs, cs;
    int softplus;
    // the grid: slots (a sequence, or a segment of one) by parts of their heads
    int slots, parts, per;
    // segments of a sequence (of one length; 1: whole) and chunks of each; by an index that a
    // segment of a cut sequence has, the state that it starts from [.., H, dk, dv] and the
    // logarithm of its whole decay [.., H]
    int segs, seg_chunks, few;  // few: up to so many segments, each forms its start itself
    float* starts;
    double* logs;
    // packed sequences that are cut: what split_kernel found
    const struct Split* split;
};

// Packed sequences cut into segments of seg_chunks chunks: the pieces in the order in which they
// are walked, longest first; those of them whose end state the next segment needs; and the
// sequences for join_kernel.  The arrays follow one another behind this header.
struct Piece {
    int n, seg, index, count;  // sequence, segment, index of its state (-1: uncut); the sequence's segments
};
struct Split {
    int pieces, ends, cuts, pad;
    int64_t ends_at, cuts_at;  // places among the Piece records behind the header
    __device__ const Piece* list(int64_t at) const { return reinterpret_cast<const Piece*>(this + 1) + at; }
};

// Workgroups go to the eight XCDs in turn, and each XCD has an L2 of its own.  A unit, the heads
// of one part of a slot, stays on one XCD, whose L2 then holds the b and c that the unit
// shares.  False: this workgroup has no unit.
__device__ __forceinline__ bool unit_of(const Params& a, int* slot, int* head) {
    const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
    const int unit = (idx / a.per) * 8 + xcd;
    if (unit >= a.slots * a.parts) return false;
    *slot = unit / a.parts;
    *head = (unit % a.parts) * a.per + idx % a.per;
    return true;
}

__device__ __forceinline__ U4 bload16(__amdgpu_buffer_rsrc_t r, int off) {
    return __builtin_bit_cast(U4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
// four values as T at a byte offset, dropped past the resource's end
template <typename T>
__device__ __forceinline__ void bstore4(__amdgpu_buffer_rsrc_t r, int off, const float (&f)[4]) {
    typedef T V __attribute__((ext_vector_type(4)));
    V v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = from_f32<T>(f[e]);
    typedef uint32_t U2 __attribute__((ext_vector_type(2)));
    if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(U2, v), r, off, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(U4, v), r, off, 0, 0);
}

// A workgroup of four waves walks CW state columns of one sequence, 16 PT of them a wave, chunk by
// chunk: one head of 128 columns, half of one, two of 64 that share b and c (HP; c . b is then
// formed once for both), or one of 64.  Wave w holds its state columns in accumulators (rows n of all of them),
// computes its share of M's ten 16 x 16 tiles into LDS, and forms y^T (columns by tokens) and the
// next state for its columns.  Two tiles of columns a wave halve the LDS reads of b, c and M, which
// at one tile took as long as the products.  The next chunk's inputs are loaded into registers
// meanwhile, through buffer resources that end with the sequence: rows behind it read as zeros, and
// their y is dropped.
// A wave's chunk (dk = 128, 32 columns) is 152 matrix instructions of 16 cycles, 96 of them the
// state's three planes, and 743 vector ones.  8 x 4096 tokens of 16 heads of 128 x 128 in bf16: 138 us
// of this pass and 63 of the pass for ENDS under a profiler, 175 in all without one (1.7 TB/s; the
// inputs and outputs alone would take 61).  No unit is full: matrix 27% and vector 33% of the cycles,
// LDS 20%.  Two waves a SIMD, which is what the registers allow, wait to issue 38% of their cycles and
// for data and the three barriers of a chunk 22%.  Eight waves a workgroup spilled (269); 64 columns a
// workgroup repeat c . b and M (195; they are for calls that leave compute units idle); with 64
// columns and four more waves that only load and form M, one barrier a chunk, this pass took 171 and
// ENDS 55.
// ENDS: the state alone, from zero, over each of a sequence's segments but the last; it goes to
// the next segment's place in `starts`, the segment's decay to `logs`.
constexpr int NW = 4;
// A sequence of up to so many segments needs no join: each segment reads the ends before it and forms
// its own start.  That is more to read with each segment (4 of 8 x 4096 tokens: 183 us without the
// join, 187 with it; 6 of 2 x 333 tokens in fp32: 15 and 17; 32 of one of 32768: 216 and 190; on the
// GPU alone, as the figures of the plans below).
constexpr int kFew = 6;
template <typename T, int DK, int DV, int CW, bool ENDS>
__global__ __launch_bounds__(64 * NW, (sizeof(T) == 2 ? NW / 2 : NW / 4)) void chunk_kernel(Params a) {
    constexpr int HP = CW > DV ? CW / DV : 1, PT = CW / (16 * NW), NTH = 64 * NW, ES = (int)sizeof(T);
    typedef Tile<T, DK, kCols> TB;
    typedef Tile<T, DK, kRows> TC;
    typedef Tile<T, CW, kBoth> TX;
    typedef typename Pair<T>::Cum Cum;
    constexpr int NB = Q * TB::UPR / NTH, NX = Q * TX::UPR / NTH;  // 16-byte units per thread
    constexpr int NT = DK / 16, KS = DK / 32;
    __shared__ __attribute__((aligned(16))) T sB[Q * DK], sC[ENDS ? 8 : Q * DK], sX[Q * CW];
    __shared__ __attribute__((aligned(16))) T sM[ENDS ? 1 : HP][ENDS ? 8 : 4 * 2 * 64 * 8];
    __shared__ __attribute__((aligned(16))) Cum sCum[AHEAD][HP][Q];
    __shared__ __attribute__((aligned(16))) float sDt[AHEAD][HP][Q], sW[AHEAD][HP][Q];

    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, l16 = lane & 15;
    const int g4 = (lane >> 4) * 4;
    int slot, hb;
    if (!unit_of(a, &slot, &hb)) return;
    const int h0 = hb * CW / DV, hw = w * 16 * PT / DV;  // the first head, this wave's among them
    const int col0 = CW < DV ? hb * CW % DV : 0;         // of a head in parts: the first column
    const int c0 = w * 16 * PT;                     // its first column of the workgroup's
    static_assert(sizeof(sB) >= (kMaxSort + 1) * sizeof(int), "scratch of longest_first");
    int n, seg = 0, index = -1, count = 1;  // index: of this segment's state, where its sequence is cut
    if (a.split) {
        if (slot >= (ENDS ? a.split->ends : a.split->pieces)) return;
        const Piece piece = a.split->list(ENDS ? a.split->ends_at : 0)[slot];
        if (piece.n < 0) return;
        n = piece.n;
        seg = piece.seg;
        index = piece.index;
        count = piece.count;
    } else if (a.cu) {
        n = __builtin_amdgcn_readfirstlane(longest_first(a.cu, a.N, slot, (int)a.T, reinterpret_cast<int*>(sB)));
    } else {
        const int steps = ENDS ? a.segs - 1 : a.segs;  // slots of a sequence
        n = slot / steps;
        seg = slot % steps;
        if (a.segs > 1) index = n * a.segs + seg;
        count = a.segs;
    }
    int64_t lo = n * a.T, hi = lo + a.T;
    if (a.cu) {
        lo = min(max(a.cu[n], (int64_t)0), a.T);
        hi = min(max(a.cu[n + 1], lo), a.T);
    }
    const int64_t end = hi;  // of the sequence
    if (index >= 0) {
        lo += (int64_t)seg * a.seg_chunks * Q;
        hi = min(hi, lo + (int64_t)a.seg_chunks * Q);
    }
    const int len = (int)(hi - lo), nc = (len + Q - 1) / Q;
    const int group = h0 / (a.H / a.G);
    const T* gx = (const T*)a.x + lo * a.xs + h0 * DV + col0;
    const T* gb = (const T*)a.b + lo * a.bs + group * DK;
    const T* gc = (const T*)a.c + lo * a.cs + group * DK;
    const T* gt = (const T*)a.dt + lo * a.dts + h0;
    T* gy = (T*)a.y + (lo * a.H + h0) * DV + col0;
    const int ys = a.H * DV;
    const float D = a.D ? a.D[h0 + hw] : 0.f;

    f32x4 S[PT][NT];  // rows 16 nt + 4g + r, column c0 + 16 pt + lane % 16
    const int64_t state = (int64_t)n * a.H + h0 + hw;
    const int at0 = g4 * DV + col0 + c0 % DV + l16;
    const float* from = a.s0 ? a.s0 + state * (DK * DV) : nullptr;
    const bool own = index >= 0 && count <= a.few;  // the start is formed here
    if (ENDS) from = nullptr;
    else if (index >= 0 && !own) from = a.starts + ((int64_t)index * a.H + h0 + hw) * (DK * DV);
    // through a resource, the rows as scalar offsets: with an address a row the registers spilled
    const auto qs = cb::buffer_over(from, DK * DV * 4);
#pragma unroll
    for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[pt][nt][r] = from ? __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                          qs, (at0 + pt * 16) * 4, (nt * 16 + r) * DV * 4, 0)) : 0.f;
    if (!ENDS && own)
        for (int e = index - seg; e < index; ++e) {
            const float keep = exp_of(a.logs[(int64_t)e * a.H + h0 + hw]);
            const auto qe = cb::buffer_over(a.starts + ((int64_t)(e + 1) * a.H + h0 + hw) * (DK * DV), DK * DV * 4);
#pragma unroll
            for (int pt = 0; pt < PT; ++pt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        S[pt][nt][r] = S[pt][nt][r] * keep +
                                       __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                           qe, (at0 + pt * 16) * 4, (nt * 16 + r) * DV * 4, 0));
        }
    // halves of M's operands that no tile writes: tiles above the diagonal
    if (!ENDS && w < HP) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sM[w][((0 * 2 + 0) * 64 + lane) * 8 + 4 + e] = from_f32<T>(0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) sM[w][((2 * 2 + 1) * 64 + lane) * 8 + 4 + e] = from_f32<T>(0.f);
    }

    U4 rb[NB], rc[NB], rx[NX];
    const int oy0 = (l16 * ys + c0 + g4) * ES;  // y of a lane's first tile
    auto load = [&](int ch) {
        const int64_t t0 = (int64_t)ch * Q;
        const int rows = min(len - ch * Q, Q);
        const auto qb = cb::buffer_over(gb + t0 * a.bs, rows * a.bs * ES);
        const auto qc = cb::buffer_over(gc + t0 * a.cs, rows * a.cs * ES);
        const auto qx = cb::buffer_over(gx + t0 * a.xs, rows * a.xs * ES);
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int id = tid + NTH * k, row = id / TB::UPR, u = id % TB::UPR;
            rb[k] = bload16(qb, row * a.bs * ES + u * 16);
            if constexpr (!ENDS) rc[k] = bload16(qc, row * a.cs * ES + u * 16);
        }
#pragma unroll
        for (int k = 0; k < NX; ++k) {
            const int id = tid + NTH * k, row = id / TX::UPR, u = id % TX::UPR;
            rx[k] = bload16(qx, row * a.xs * ES + u * 16);
        }
    };
    // Decays of the four chunks from ch on, a chunk a wave, a token a lane: a token behind the end
    // decays and adds nothing.  One wave at a time forming the next chunk's kept the others waiting
    // for 2000 of 14000 cycles.  The raw time steps are loaded a chunk before they are needed, and
    // carried as they are: widening them would wait for them.
    T rdt[HP];
    auto load_dt = [&](int ch) {
        const int t = min((ch + w) * Q + lane, len - 1);
#pragma unroll
        for (int hp = 0; hp < HP; ++hp) rdt[hp] = gt[(int64_t)t * a.dts + hp];
    };
    double logs[HP] = {};  // ENDS: this wave's part of the logarithms of the segment's decays
    auto decays = [&](int ch) {
        const int k = (ch + w) % AHEAD;
#pragma unroll
        for (int hp = 0; hp < HP; ++hp) {
            const float bias = a.dt_bias ? a.dt_bias[h0 + hp] : 0.f;
            const float dt = (ch + w) * Q + lane < len ? time_step(to_f32(rdt[hp]) + bias, a.softplus) : 0.f;
            const double cum = scan(log_decay(dt, a.A[h0 + hp])), all = last_lane(cum);
            if constexpr (ENDS) logs[hp] += all;
            sCum[k][hp][lane] = Pair<T>::cum(cum);
            sDt[k][hp][lane] = dt;
            sW[k][hp][lane] = exp_of(all - cum) * dt;
        }
    };
    const int stB = TB::at(tid / TB::UPR, tid % TB::UPR * TB::EPU), stC = TC::at(tid / TB::UPR, tid % TB::UPR * TB::EPU);
    const int stX = TX::at(tid / TX::UPR, tid % TX::UPR * TX::EPU);
    // a thread's unit k lies k NTH units on: as many rows below, whose swizzle differs by that of
    // the rows between
    constexpr int RB = NTH / TB::UPR, RX = NTH / TX::UPR;
    auto put = [](void* tile, int base, int swz, int k, const U4& v) {
        *reinterpret_cast<U4*>(static_cast<char*>(tile) + (base ^ (swz << 4)) + k * NTH * 16) = v;
    };
    auto store = [&]() {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            put(sB, stB, TB::swz(k * RB), k, rb[k]);
            if constexpr (!ENDS) put(sC, stC, TC::swz(k * RB), k, rc[k]);
        }
#pragma unroll
        for (int k = 0; k < NX; ++k) put(sX, stX, TX::swz(k * RX), k, rx[k]);
    };
    const int bRowsB = rows_base<TB>(lane), bRowsC = rows_base<TC>(lane), bPermC = perm_base<TC>(lane);
    const int bColsB = cols_base<TB, T>(lane), bColsX = cols_base<TX, T>(lane), bPermX = perm_base<TX>(lane);
    if (nc > 0) {
        load_dt(0);
        load(0);
        decays(0);
        store();
    }
    for (int ch = 0; ch < nc; ++ch) {
        const int k = ch % AHEAD;
        cb::lds_barrier();  // the chunk is in LDS
        // loads return in order: a wait for the time steps must not be one for the next chunk
        if (ch % 4 == 2) load_dt(ch + 2);
        if (ch + 1 < nc) load(ch + 1);
        const int rowsB = fresh(bRowsB), rowsC = fresh(bRowsC), permC = fresh(bPermC), colsB = fresh(bColsB), permX = fresh(bPermX);
        f32x4 Y[PT][4];
        // Every stage reads the next one's operands before its own products, and carries as much
        // vector work of another stage as its products leave issue slots for; the fences keep the
        // compiler from gathering either.
        if constexpr (!ENDS) {
            // M's ten tiles (it, jt), jt <= it, three a wave (two of them twice)
            const int its = w == 0 ? 0x033 : w == 1 ? 0x133 : w == 2 ? 0x222 : 0x111;
            const int jts = w == 0 ? 0x010 : w == 1 ? 0x032 : w == 2 ? 0x210 : 0x111;
            int ob[3], oc[3];
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                ob[t] = rowsB + (jts >> (4 * t) & 15) * 16 * TB::RB;
                oc[t] = rowsC + (its >> (4 * t) & 15) * 16 * TC::RB;
            }
            f32x4 G[3] = {zero4(), zero4(), zero4()};
            Frag<T> gb_[2][3], gc_[2][3], fc[2][4];
            auto read_g = [&](int s) {
#pragma unroll
                for (int t = 0; t < 3; ++t) {
                    gb_[s & 1][t] = rows_contig<TB>(sB, ob[t], 0, s * 32);
                    gc_[s & 1][t] = rows_contig<TC>(sC, oc[t], 0, s * 32);
                }
            };
            auto read_c = [&](int s) {
#pragma unroll
                for (int it = 0; it < 4; ++it) fc[s & 1][it] = rows_perm<TC, T>(sC, permC, it * 16, s * 32);
            };
            read_g(0);
            cb::sched_fence();
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                if (s + 1 < KS) read_g(s + 1);
                else read_c(0);
                cb::sched_fence();
#pragma unroll
                for (int t = 0; t < 3; ++t) mma(G[t], gb_[s & 1][t], gc_[s & 1][t]);
                cb::sched_fence();
            }
            // what the entering state gives: y^T[p, i] = exp(cum_i) sum_n S[n, p] c[i, n]
#pragma unroll
            for (int pt = 0; pt < PT; ++pt)
#pragma unroll
                for (int it = 0; it < 4; ++it) Y[pt][it] = zero4();
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                if (s + 1 < KS) read_c(s + 1);
                // In bf16 one plane of S here, and of M below: with both y is off by 5e-4 of its size (RMS)
                // before its own rounding, which is 17e-4.  Two planes would be 44 matrix instructions
                // more of 152.  S itself keeps fp32.
                Frag<T> fs[PT];
#pragma unroll
                for (int pt = 0; pt < PT; ++pt) fs[pt] = frag_from_acc<T>(S[pt][2 * s], S[pt][2 * s + 1]);
                cb::sched_fence();
#pragma unroll
                for (int it = 0; it < 4; ++it)
#pragma unroll
                    for (int pt = 0; pt < PT; ++pt) mma(Y[pt][it], fs[pt], fc[s & 1][it]);
                // a tile of M beside them
#pragma unroll
                for (int t = s * 3 / KS; t < (s + 1) * 3 / KS; ++t) {
                    const int it = its >> (4 * t) & 15, jt = jts >> (4 * t) & 15, i = it * 16 + l16, j = jt * 16 + g4;
#pragma unroll
                    for (int hp = 0; hp < HP; ++hp) {
                        const Cum ci = sCum[k][hp][i];
                        const Vec<Cum, 4> cj = load_vec<Cum, 4>(&sCum[k][hp][j]);
                        const Vec<float, 4> dj = load_vec<float, 4>(&sDt[k][hp][j]);
                        typedef T V __attribute__((ext_vector_type(4)));
                        V m;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float v = G[t][r] * Pair<T>::decay(ci, cj.v[r]) * dj.v[r];
                            m[r] = from_f32<T>(j + r <= i ? v : 0.f);
                        }
                        *reinterpret_cast<V*>(&sM[hp][((it * 2 + (jt >> 1)) * 64 + lane) * 8 + (jt & 1) * 4]) = m;
                    }
                }
                cb::sched_fence();
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const float e = Pair<T>::decay(sCum[k][hw][it * 16 + l16]);
#pragma unroll
                for (int pt = 0; pt < PT; ++pt) Y[pt][it] *= e;
            }
            cb::lds_barrier();  // M is in LDS
        }
        Frag<T> fx[PT][2], fb[3];
        float wt[2][8];
        Planes<T> wx[2][PT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) fx[pt][s] = cols_perm<TX>(sX, bColsX, s * 32, c0 + pt * 16);
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const Vec<float, 4> v = load_vec<float, 4>(&sW[k][hw][s * 32 + e * 4 + g4]);
#pragma unroll
                for (int r = 0; r < 4; ++r) wt[s][e + r] = v.v[r];
            }
        }
        // pair u of the 4 PT pairs of weighted x that tokens 32 s on need
        auto plane = [&](int s, int u) { wx[s][u / 4].set(fx[u / 4][s], u % 4 * 2, wt[s][u % 4 * 2], wt[s][u % 4 * 2 + 1]); };
        const int rows = min(len - ch * Q, Q);
        const auto qy = cb::buffer_over(gy + (int64_t)ch * Q * ys, rows * ys * ES);
        const int oy = fresh(oy0);
        Vec<T, 4> xq[2];
        auto read_x = [&](int u) { xq[u & 1] = lds_vec<T, 4>(sX, permX ^ ((c0 + u % PT * 16) * ES + u / PT * 16 * TX::RB)); };
        auto put_y = [&](int u) {
            const int it = u / PT, pt = u % PT;
            float o[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = Y[pt][it][r] + D * to_f32(xq[u & 1].v[r]);
            bstore4<T>(qy, oy + (it * 16 * ys + pt * 16) * ES, o);
        };
        const float gone = Pair<T>::decay(sCum[k][hw][Q - 1]);
        auto read_b = [&](int u) { fb[u % 3] = cols_perm<TB>(sB, colsB, u / NT * 32, u % NT * 16); };
        if constexpr (!ENDS) {
            // the chunk's own part: six pieces of M, with the first half's planes beside them
            Frag<T> fm[2];
            auto read_m = [&](int u) {
                const int it = u < 2 ? u : u < 4 ? 2 : 3, s = u < 2 ? 0 : u & 1;
                const Vec<T, 8> v = load_vec<T, 8>(&sM[hw][((it * 2 + s) * 64 + lane) * 8]);
#pragma unroll
                for (int e = 0; e < 8; ++e) fm[u & 1].v[e] = v.v[e];
            };
            float odd = 0.f;
            read_m(0);
            read_x(0);
            read_x(1);
            cb::sched_fence();
#pragma unroll
            for (int u = 0; u < 6; ++u) {
                const int it = u < 2 ? u : u < 4 ? 2 : 3, s = u < 2 ? 0 : u & 1;
                if (u < 5) read_m(u + 1);
                cb::sched_fence();
#pragma unroll
                for (int pt = 0; pt < PT; ++pt) mma(Y[pt][it], fx[pt][s], fm[u & 1]);
#pragma unroll
                for (int v = u * 4 * PT / 6; v < (u + 1) * 4 * PT / 6; ++v) plane(0, v);
                cb::sched_fence();
                // y of the 16 tokens whose last piece was the one before
                const int done = u == 1 ? 0 : u == 2 ? 1 : u == 4 ? 2 : -1;
                if (done >= 0) {
#pragma unroll
                    for (int v = done * PT; v < done * PT + PT; ++v) {
                        put_y(v);
                        if (v + 2 < 4 * PT) read_x(v + 2);
                    }
                }
                if (done == 2) {
#pragma unroll
                    for (int pt = 0; pt < PT; ++pt)
#pragma unroll
                        for (int r = 0; r < 4; ++r) odd = fmaf(0.f, Y[pt][2][r], odd);
                }
            }
#pragma unroll
            for (int v = 3 * PT; v < 4 * PT; ++v) {
                put_y(v);
                if (v + 2 < 4 * PT) read_x(v + 2);
            }
            read_b(0);
            read_b(1);
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) wx[0][pt].formed();  // beside the products above
            // M times x takes an x that is not finite to the tokens before it too: 0 x inf.  Tokens 32 to 47
            // have met all of the chunk's x, so there it shows.  y once more, a tile at a time, with zeros in
            // the place of such x, and NaN in its column from its token on.  Looking for it costs 2% of a
            // call (8 x 4096 tokens of 16 heads of 128 x 128: 171 and 175 us).
            if (__builtin_expect(__builtin_amdgcn_ballot_w64(odd != odd) != 0, 0)) {
#pragma unroll 1
                for (int it = 0; it < 4; ++it) {
#pragma unroll
                    for (int pt = 0; pt < PT; ++pt) {
                        cb::sched_fence();
                        const int ln = fresh(lane), l16 = ln & 15, g4 = (ln >> 4) * 4;
                        const int permC = perm_base<TC>(ln), colsX = cols_base<TX, T>(ln);
                        f32x4 y = zero4();
#pragma unroll
                        for (int s = 0; s < KS; ++s) {
                            f32x4 lo = S[pt][2 * s], hi = S[pt][2 * s + 1];
                            asm volatile("" : "+v"(lo), "+v"(hi));  // not converted for all of the tiles at once
                            mma(y, frag_from_acc<T>(lo, hi), rows_perm<TC, T>(sC, permC, it * 16, s * 32));
                            cb::sched_fence();
                        }
                        y *= Pair<T>::decay(sCum[k][hw][it * 16 + l16]);
                        for (int s = 0; s <= it >> 1; ++s) {
                            Frag<T> x = cols_perm<TX>(sX, colsX, s * 32, c0 + pt * 16), m;
                            const Vec<T, 8> v = load_vec<T, 8>(&sM[hw][((it * 2 + s) * 64 + ln) * 8]);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                m.v[e] = v.v[e];
                                x.v[e] = is_finite(to_f32(x.v[e])) ? x.v[e] : from_f32<T>(0.f);
                            }
                            mma(y, x, m);
                        }
#pragma unroll 1
                        for (int j = 0; j < it * 16 + 16; ++j) {
                            const Vec<T, 4> x = lds_vec<T, 4>(sX, TX::at(j, c0 + pt * 16 + g4));
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (!is_finite(to_f32(x.v[r])) && j <= it * 16 + l16) y[r] = __uint_as_float(__float_as_uint(y[r]) | 0x7fc00000u);
                        }
                        const Vec<T, 4> x = lds_vec<T, 4>(sX, TX::at(it * 16 + l16, c0 + pt * 16 + g4));
                        float o[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[r] = y[r] + D * to_f32(x.v[r]);
                        bstore4<T>(qy, ((it * 16 + l16) * ys + c0 + pt * 16 + g4) * ES, o);
                    }
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < 4 * PT; ++v) plane(0, v);
            read_b(0);
            read_b(1);
        }
        // the next state, a tile of rows at a time
        auto scale = [&](int nt) {
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) S[pt][nt] *= gone;
        };
        scale(0);
        cb::sched_fence();
#pragma unroll
        for (int u = 0; u < 2 * NT; ++u) {
            const int s = u / NT, nt = u % NT;
            if (u + 2 < 2 * NT) read_b(u + 2);
            cb::sched_fence();
#pragma unroll
            for (int i = 0; i < Planes<T>::N; ++i)
#pragma unroll
                for (int pt = 0; pt < PT; ++pt) mma(S[pt][nt], fb[u % 3], wx[s][pt].p[i]);
            if (s == 0) {
                if (nt + 1 < NT) scale(nt + 1);
#pragma unroll
                for (int v = nt * 4 * PT / NT; v < (nt + 1) * 4 * PT / NT; ++v) plane(1, v);
            }
            cb::sched_fence();
        }
        cb::lds_barrier();  // the chunk has been read
        if (ch % 4 == 3) decays(ch + 1);
        if (ch + 1 < nc) store();
    }
    float* to = nullptr;
    if (ENDS) to = a.starts + ((int64_t)(index + 1) * a.H + h0 + hw) * (DK * DV);
    else if (a.sT && hi == end) to = a.sT + state * (DK * DV);
    if (to) {
        const auto qt = cb::buffer_over(to, DK * DV * 4);
#pragma unroll
        for (int pt = 0; pt < PT; ++pt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, (float)S[pt][nt][r]), qt,
                                                          (at0 + pt * 16) * 4, (nt * 16 + r) * DV * 4, 0);
    }
    if constexpr (ENDS) {
        __shared__ double sLogs[HP][NW];
#pragma unroll
        for (int hp = 0; hp < HP; ++hp)
            if (lane == 0) sLogs[hp][w] = logs[hp];
        __syncthreads();
        if (tid < HP && col0 == 0) a.logs[(int64_t)index * a.H + h0 + tid] = (sLogs[tid][0] + sLogs[tid][1]) + (sLogs[tid][2] + sLogs[tid][3]);
    }
}

// For the segments of a sequence cut into more than a.few: starts[0] = the initial state, starts[s + 1]
// = exp(logs[s]) starts[s] + the segment's own end, which is in starts[s + 1].  The forward pass
// reads every segment's start from here, so it may write the final state over the initial one (for
// a call that does, a.few is 0).
__global__ __launch_bounds__(256) void join_kernel(Params a, int dk) {
    const int64_t quads = (int64_t)dk * a.dv / 4, row = quads * a.H;  // r: place in a sequence's states
    const int64_t all = (a.split ? a.split->cuts : a.N) * row;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < all; id += (int64_t)gridDim.x * 256) {
        const int64_t j = id / row, r = id % row;
        int n = (int)j, base = n * a.segs, segs = a.segs;
        if (a.split) {
            const Piece cut = a.split->list(a.split->cuts_at)[j];
            n = cut.n;
            base = cut.index;
            segs = cut.count;
        }
        f32x4* st = reinterpret_cast<f32x4*>(a.starts) + base * row + r;
        const double* lg = a.logs + (int64_t)base * a.H + r / quads;
        f32x4 s = a.s0 ? reinterpret_cast<const f32x4*>(a.s0)[n * row + r] : zero4();
        st[0] = s;
        constexpr int AT = 4;  // segments whose ends are loaded together
        for (int g = 0; g + 1 < segs; g += AT) {
            f32x4 own[AT];
            double l[AT];
#pragma unroll
            for (int k = 0; k < AT; ++k) {
                const int at = min(g + k, segs - 2);
                own[k] = st[(int64_t)(at + 1) * row];
                l[k] = lg[(int64_t)at * a.H];
            }
#pragma unroll
            for (int k = 0; k < AT; ++k) {
                if (g + k + 1 >= segs) break;
                s = s * exp_of(l[k]) + own[k];
                st[(int64_t)(g + k + 1) * row] = s;
            }
        }
    }
}

// The pieces of packed sequences, sorted by their chunks through a histogram; one workgroup.  The
// lists hold max_ends ends of segments, more than sequences side by side in the token axis can have;
// where offsets overlap, sequences past them are left whole.  index_of [N] holds a cut sequence's
// first state, -1 for the others.
constexpr int kBins = 2048;  // more than a segment's chunks
__global__ __launch_bounds__(1024) void split_kernel(const int64_t* __restrict__ cu, int N, int64_t total, int seg_chunks,
                                                     Split* split, int max_ends, int64_t ends_at, int64_t cuts_at,
                                                     int* index_of, int few) {
    __shared__ int at[kBins];  // first pieces of a size: a count, then the place of the next one
    __shared__ int sums[1024];
    __shared__ unsigned long long ends;  // with the ends given back: of 2^23 sequences that overlap more than 2^32
    __shared__ int cuts, states;
    const int tid = threadIdx.x;
    Piece* list = reinterpret_cast<Piece*>(split + 1);
    at[tid] = at[tid + 1024] = 0;
    if (tid == 0) {
        ends = 0;
        cuts = states = 0;
    }
    __syncthreads();
    auto chunks = [&](int n) {
        const int64_t lo = min(max(cu[n], (int64_t)0), total), hi = min(max(cu[n + 1], lo), total);
        return (int)((hi - lo + Q - 1) / Q);
    };
    auto bin = [](int c) { return min(c, kBins - 1); };
    // a sequence: `full` whole segments and a piece of the rest, or one piece
    for (int n = tid; n < N; n += 1024) {
        const int c = chunks(n), full = c / seg_chunks, rest = c - full * seg_chunks, segs = full + (rest ? 1 : 0);
        int index = -1;
        if (segs > 1) {
            const int64_t e = (int64_t)atomicAdd(&ends, (unsigned long long)(segs - 1));
            if (e + segs - 1 <= max_ends) {
                index = atomicAdd(&states, segs);
                for (int k = 0; k + 1 < segs; ++k) list[ends_at + e + k] = Piece{n, k, index + k, segs};
                if (segs > few) list[cuts_at + atomicAdd(&cuts, 1)] = Piece{n, 0, index, segs};
                atomicAdd(&at[seg_chunks], full);
                if (rest) atomicAdd(&at[rest], 1);
            } else {  // given back as ends of nothing
                for (int k = 0; k + 1 < segs && e + k < max_ends; ++k) list[ends_at + e + k] = Piece{-1, 0, 0, 0};
            }
        }
        if (index < 0) atomicAdd(&at[bin(c)], 1);
        index_of[n] = index;
    }
    __syncthreads();
    // sizes from the largest down: thread t has the bin kBins - 1 - 2t and the one below
    const int hi = kBins - 1 - 2 * tid, a = at[hi], b = at[hi - 1];
    sums[tid] = a + b;
    __syncthreads();
    for (int d = 1; d < 1024; d <<= 1) {
        const int v = tid >= d ? sums[tid - d] : 0;
        __syncthreads();
        sums[tid] += v;
        __syncthreads();
    }
    const int before = sums[tid] - a - b;
    at[hi] = before;
    at[hi - 1] = before + a;
    const int pieces = sums[1023];
    __syncthreads();
    for (int n = tid; n < N; n += 1024) {
        const int c = chunks(n), index = index_of[n];
        if (index < 0) {
            list[atomicAdd(&at[bin(c)], 1)] = Piece{n, 0, -1, 1};
            continue;
        }
        const int full = c / seg_chunks, rest = c - full * seg_chunks, segs = full + (rest ? 1 : 0);
        const int p = atomicAdd(&at[seg_chunks], full);
        for (int k = 0; k < full; ++k) list[p + k] = Piece{n, k, index + k, segs};
        if (rest) list[atomicAdd(&at[rest], 1)] = Piece{n, full, index + full, segs};
    }
    if (tid == 0) *split = Split{pieces, (int)min((int64_t)ends, (int64_t)max_ends), cuts, 0, ends_at, cuts_at};
}

Params params(const SsmArgs& a) {
    return Params{a.x, a.dt, a.b, a.c, a.A, a.D, a.dt_bias, a.initial_state, a.y, a.final_state, a.cu_seqlens, a.T,
                  (int)a.N, (int)a.H, (int)a.G, (int)a.dv, (int)a.x_stride, (int)a.dt_stride, (int)a.b_stride,
                  (int)a.c_stride, a.softplus ? 1 : 0, 0, 0, 0, 1, 0, 0, nullptr, nullptr, nullptr};
}

// Parts of a slot's `blocks` workgroups: the fewest that leave the eight XCDs with about as many units each (at
// most an eighth more than their share).
void set_grid(Params* p, int slots, int blocks) {
    p->slots = slots;
    p->parts = blocks;
    for (int k = 1; k < blocks; ++k) {
        if (blocks % k) continue;
        const int64_t units = (int64_t)slots * k;
        if ((units + 7) / 8 * 64 <= units * 9) {
            p->parts = k;
            break;
        }
    }
    p->per = blocks / p->parts;
}
unsigned grid_of(const Params& p) { return (unsigned)(((int64_t)p.slots * p.parts + 7) / 8 * 8 * p.per); }

// How a call is cut, and its workspace.
struct Plan {
    int segs, seg_chunks;                 // as Params; packed: segs 0, cut by split_kernel
    int64_t indexes, pieces, ends, cuts;  // at most: states of segments; packed: pieces and lists
    int64_t starts, logs, split, index_of, total;  // byte offsets of the workspace, its size (0: none)
};

// Sequences of one length.  A chunk's time is the unit.  A compute unit runs two workgroups (of 128
// state columns) at once, each then 1.36 times as long as one alone; halves of heads take 0.65 of it;
// the pass for the segments' ends takes half a chunk's time a chunk; launches, the states' way through
// HBM and the join, which walks the segments, are the rest.  Fitted to calls; now in us, the chosen one
// first: 128 sequence-heads of 64 chunks in 4 / 1 (halves) / 2 / 3 / 8 segments 183 / 201 / 208 / 182 /
// 197; 16 of 512 in 32 / 16 / 48 190 / 219 / 189; 8 of 32 in 16 / 8 / 32 26 / 29 / 36, in whole heads 31 /
// 37 / 36; fp32, whose chunks take three times as long, 18 of 11 in 6 / 3 / 11 39 / 56 / 44.
Plan plan_fixed(int64_t N, int64_t T, int64_t H, int64_t dk, int64_t dv, bool bf16_in, int64_t cus) {
    Plan p{};
    const int64_t nc = (T + Q - 1) / Q, heads = N * H;
    // workgroups of a segment: pairs of heads of 64 columns only where there are enough of them
    const int64_t chains = dv == 128 || heads <= cus ? heads : (heads + 1) / 2;
    auto rounds = [&](int64_t w) {
        if (dv == 128 && 2 * w <= cus) return 0.65;  // heads in halves
        return w <= cus ? 1.0 : 1.36 * (double)((w + 2 * cus - 1) / (2 * cus));
    };
    double best = rounds(chains) * (double)nc;
    p.segs = 1;
    for (int64_t g = 2; g <= nc && g <= 128 && chains * g <= 8 * cus; ++g) {
        const int64_t len = (nc + g - 1) / g;
        if ((nc + len - 1) / len != g) continue;
        const double rest = (g > kFew ? 3.0 + 0.06 * (double)g : 2.0) + 0.009 * (double)(chains * g);
        const double cost = rounds(chains * g) * (double)len + 0.5 * rounds(chains * (g - 1)) * (double)len +
                            (bf16_in ? rest : 0.3 * rest);
        if (cost < best) {
            best = cost;
            p.segs = (int)g;
        }
    }
    p.seg_chunks = (int)((nc + p.segs - 1) / p.segs);
    if (p.segs > 1) {
        p.indexes = N * p.segs;
        p.logs = p.indexes * H * dk * dv * 4;
        p.total = p.logs + (p.indexes * H * 8 + 255) / 256 * 256;
    }
    return p;
}

// Packed sequences, whose lengths the host does not know: segments of as many chunks as a workgroup
// slot of the GPU has of all, or two thirds of it where there are sequences enough to fill the slots
// (then only the longest are cut, and the launch does not wait for their chains alone); at least
// four, in fp32, whose chunks outweigh a segment's costs, two.  In us, segments of the rule / half as
// long / whole sequences: 16 prompts of about 700 tokens, 16 heads 148 / 153 / 247; 64 of 512, 32 heads
// of 64 columns 279 / 301 / 333; 8 of 300, 6 heads in fp32 36 / - / 206 (segments of four 47).
Plan plan_packed(int64_t N, int64_t total, int64_t H, int64_t dk, int64_t dv, bool bf16_in, int64_t cus) {
    Plan p{};
    p.segs = 1;
    const int64_t nc = total / Q + N, wide = H * dv < 128 ? 1 : H * dv / 128, slots = N * wide < 2 * cus ? 2 * cus : 3 * cus;
    const int64_t least = bf16_in ? 4 : 2;
    int64_t len = (nc * wide + slots - 1) / slots;
    if (len < least) len = least;
    if (len > kBins - 1) len = kBins - 1;
    if (total <= len * Q) return p;  // no sequence can be longer than a segment
    p.segs = 0;
    p.seg_chunks = (int)len;
    // a cut sequence of k segments has more than (k - 1) len chunks' tokens
    p.ends = total / (len * Q);
    p.cuts = p.ends;
    p.pieces = p.ends + N;
    p.indexes = 2 * p.ends;
    p.logs = p.indexes * H * dk * dv * 4;
    p.split = p.logs + (p.indexes * H * 8 + 255) / 256 * 256;
    p.index_of = p.split + (int64_t)sizeof(Split) + (p.pieces + p.ends + p.cuts) * (int64_t)sizeof(Piece);
    p.total = (p.index_of + N * 4 + 255) / 256 * 256;
    return p;
}

template <typename T, int DK, int DV, int CW>
hipError_t launch_chunks(const SsmArgs& a, const Plan& plan, void* workspace) {
    Params p = params(a);
    const hipStream_t stream = (hipStream_t)a.stream;
    const int blocks = (int)a.H * DV / CW;
    char* ws = static_cast<char*>(workspace);
    int64_t ends = 0, cuts = 0, slots = a.N;
    if (plan.total) {
        p.segs = plan.segs;
        p.seg_chunks = plan.seg_chunks;
        p.starts = reinterpret_cast<float*>(ws + plan.starts);
        p.logs = reinterpret_cast<double*>(ws + plan.logs);
        // not where a final state may replace the initial one that other segments still read
        p.few = a.initial_state && a.initial_state == a.final_state ? 0 : kFew;
        if (a.cu_seqlens) {
            Split* split = reinterpret_cast<Split*>(ws + plan.split);
            p.split = split;
            hipLaunchKernelGGL(split_kernel, dim3(1), dim3(1024), 0, stream, a.cu_seqlens, (int)a.N, a.T, plan.seg_chunks,
                               split, (int)plan.ends, plan.pieces, plan.pieces + plan.ends,
                               reinterpret_cast<int*>(ws + plan.index_of), p.few);
            ends = plan.ends;
            cuts = plan.cuts;
            slots = plan.pieces;
        } else {
            ends = a.N * (plan.segs - 1);
            cuts = a.N;
            slots = a.N * plan.segs;
        }
        set_grid(&p, (int)ends, blocks);
        hipLaunchKernelGGL((chunk_kernel<T, DK, DV, CW, true>), dim3(grid_of(p)), dim3(64 * NW), 0, stream, p);
        // workgroups that fit the GPU at once: how many sequences there are to join the host does not know
        const int64_t need = (cuts * a.H * DK * DV / 4 + 255) / 256, fit = a.cus * 8;
        if ((a.cu_seqlens ? plan.ends + 1 : plan.segs) > p.few)
            hipLaunchKernelGGL(join_kernel, dim3((unsigned)(need < fit ? need : fit)), dim3(256), 0, stream, p, DK);
    }
    set_grid(&p, (int)slots, blocks);
    hipLaunchKernelGGL((chunk_kernel<T, DK, DV, CW, false>), dim3(grid_of(p)), dim3(64 * NW), 0, stream, p);
    return hipGetLastError();
}

template <typename T, int DK>
hipError_t launch_dk(const SsmArgs& a, const Plan& plan, void* ws) {
    const int64_t heads = (plan.pieces ? plan.pieces : a.N * (plan.total ? plan.segs : 1)) * a.H;
    // Heads of 128 columns go to two workgroups each while every one then has a compute unit of its own
    // (8 heads of 300 tokens 17 us, whole 23; 160 heads of 128 in fp32, which have not, 44 and 36).
    if (a.dv == 128)
        return 2 * heads <= a.cus ? launch_chunks<T, DK, 128, 64>(a, plan, ws) : launch_chunks<T, DK, 128, 128>(a, plan, ws);
    // Two heads of 64 a workgroup where a group has an even number of them and pairs still fill the
    // GPU: c . b and the staging of b and c are shared, but few workgroups take longer.
    return a.H / a.G % 2 == 0 && heads / 2 >= a.cus ? launch_chunks<T, DK, 64, 128>(a, plan, ws)
                                                     : launch_chunks<T, DK, 64, 64>(a, plan, ws);
}
template <typename T>
hipError_t launch_fwd(const SsmArgs& a, void* ws) {
    Plan plan{};
    if (ws) plan = a.cu_seqlens ? plan_packed(a.N, a.T, a.H, a.dk, a.dv, a.dtype_bf16, a.cus)
                                : plan_fixed(a.N, a.T, a.H, a.dk, a.dv, a.dtype_bf16, a.cus);
    return a.dk == 128 ? launch_dk<T, 128>(a, plan, ws) : launch_dk<T, 64>(a, plan, ws);
}

// ---- single tokens --------------------------------------------------------------------------
// As the recurrence's decode step: a workgroup owns the state of one (sequence, head), read and
// written once with 16-byte accesses; a thread holds a column quad of its rows, and y's sums over
// the rows go through LDS.  Bound by HBM.  STREAM: past the caches, for states of which two do not
// fit them together.  Such a state is not there any more when its layer's next token comes: three
// of 268 MB in turn take 96 us a step instead of 105 (one alone, which no stack of layers has, would
// take 95 instead of 80).
template <typename T, int DK, int DV, bool STREAM>
__global__ __launch_bounds__(256) void step_kernel(Params a) {
    constexpr int NQ = DV / 4, NRG = 256 / NQ, RPG = DK / NRG;
    static_assert(RPG * NRG == DK && NQ * NRG == 256, "step tiling");
    __shared__ __attribute__((aligned(16))) float sRed[NRG][DV];
    __shared__ float sB[DK], sC[DK];
    const int tid = threadIdx.x, cq = tid % NQ, rg = tid / NQ;
    const int64_t n = blockIdx.x / a.H;
    const int h = blockIdx.x % a.H, group = h / (a.H / a.G);
    float* st = a.sT + ((int64_t)blockIdx.x * DK + rg * RPG) * DV + cq * 4;
    f32x4 s[RPG];
#pragma unroll
    for (int i = 0; i < RPG; ++i) {
        const f32x4* p = reinterpret_cast<const f32x4*>(st + (int64_t)i * DV);
        if constexpr (STREAM) s[i] = __builtin_nontemporal_load(p);
        else s[i] = *p;
    }
    if (tid < DK) {
        sB[tid] = to_f32(((const T*)a.b)[n * a.bs + group * DK + tid]);
        sC[tid] = to_f32(((const T*)a.c)[n * a.cs + group * DK + tid]);
    }
    const float dt = time_step(to_f32(((const T*)a.dt)[n * a.dts + h]) + (a.dt_bias ? a.dt_bias[h] : 0.f), a.softplus);
    const float decay = expf(dt * a.A[h]);
    const Vec<T, 4> xv = load_vec<T, 4>((const T*)a.x + n * a.xs + h * DV + cq * 4);
    f32x4 dx, acc = zero4();
#pragma unroll
    for (int e = 0; e < 4; ++e) dx[e] = dt * to_f32(xv.v[e]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RPG; ++i) {
        const float b = sB[rg * RPG + i], c = sC[rg * RPG + i];
        s[i] = s[i] * decay + b * dx;
        acc += s[i] * c;
        f32x4* p = reinterpret_cast<f32x4*>(st + (int64_t)i * DV);
        if constexpr (STREAM) __builtin_nontemporal_store(s[i], p);
        else *p = s[i];
    }
    *reinterpret_cast<f32x4*>(&sRed[rg][cq * 4]) = acc;
    __syncthreads();
    if (tid < DV) {
        float o = a.D ? a.D[h] * to_f32(((const T*)a.x)[n * a.xs + h * DV + tid]) : 0.f;
#pragma unroll
        for (int r = 0; r < NRG; ++r) o += sRed[r][tid];
        ((T*)a.y)[(int64_t)blockIdx.x * DV + tid] = from_f32<T>(o);
    }
}

template <typename T, int DK, int DV>
hipError_t launch_step_t(const SsmArgs& a) {
    const bool stream = a.N * a.H * DK * DV * 4 > (int64_t)128 << 20;  // the last cache holds 256 MB
    auto kernel = stream ? step_kernel<T, DK, DV, true> : step_kernel<T, DK, DV, false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(a.N * a.H)), dim3(256), 0, (hipStream_t)a.stream, params(a));
    return hipGetLastError();
}
template <typename T>
hipError_t launch_step(const SsmArgs& a) {
    if (a.dk == 128) return a.dv == 128 ? launch_step_t<T, 128, 128>(a) : launch_step_t<T, 128, 64>(a);
    return a.dv == 128 ? launch_step_t<T, 64, 128>(a) : launch_step_t<T, 64, 64>(a);
}

}  // namespace ssm

size_t ssm_workspace_bytes(bool packed, int64_t N, int64_t T, int64_t H, int64_t dk, int64_t dv, bool bf16_in,
                           int64_t cus) {
    return (size_t)(packed ? ssm::plan_packed(N, T, H, dk, dv, bf16_in, cus) : ssm::plan_fixed(N, T, H, dk, dv, bf16_in, cus))
                        .total;
}

hipError_t launch_ssm_fwd(const SsmArgs& a, void* workspace) {
    return a.dtype_bf16 ? ssm::launch_fwd<bf16>(a, workspace) : ssm::launch_fwd<float>(a, workspace);
}

hipError_t launch_ssm_step(const SsmArgs& a) {
    return a.dtype_bf16 ? ssm::launch_step<bf16>(a) : ssm::launch_step<float>(a);
}

}  // namespace gdn2
