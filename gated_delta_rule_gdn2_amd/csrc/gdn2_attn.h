// gdn2_attn.h -- device-side building blocks of the attention kernels.
//
// Products are 32 x 32 tiles (v_mfma_f32_32x32x16_bf16, or v_mfma_f32_32x32x2_f32 for fp32 inputs)
// with fp32 accumulators.  An operand holds 16 contraction slots, 8 a lane: lane l covers row or
// column l % 32 and the slots (g, e), g = l / 32, e = 0 .. 7, in one of two maps:
//   contiguous: slot (g, e) -> 8 g + e
//   permuted:   slot (g, e) -> 8 (e / 4) + 4 g + e % 4
// An accumulator keeps rows 8 (i / 4) + 4 g + i % 4 of column l % 32 in its 16 registers i, so its
// registers 0 .. 7 and 8 .. 15 are two operands in the permuted map as they stand.  Scores are
// therefore formed with the axis that the next product sums over in the rows, and go from one
// product into the next without leaving the registers.
#pragma once

#include "gdn2_device.h"
#include "gdn2_launch.h"

namespace gdn2 {
namespace attn {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
#define GDN2_LDS __attribute__((address_space(3)))

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <typename T> struct Op;
template <> struct Op<bf16> { bf16x8 v; };
template <> struct Op<float> { float v[8]; };

__device__ __forceinline__ void mma(f32x16& c, const Op<bf16>& a, const Op<bf16>& b) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x16& c, const Op<float>& a, const Op<float>& b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[e], b.v[e], c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
    return z;
}
// registers 8 h .. 8 h + 7 of an accumulator as an operand in the permuted map
template <typename T> __device__ __forceinline__ Op<T> op_of(const f32x16& c, int h) {
    Op<T> r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = from_f32<T>(c[8 * h + e]);
    return r;
}
// the row of an accumulator's register i
__device__ __forceinline__ int acc_row(int i, int g) { return 8 * (i / 4) + 4 * g + i % 4; }

// An address in LDS, as the number it is.  Bytes are addressed by a lane's own base and constants:
// the base goes through `opaque` once a tile, or the compiler keeps every sum of the two in a register
// of its own through the loop.
typedef uint32_t Lds;
__device__ __forceinline__ Lds lds_of(const void* p) { return (Lds)(uintptr_t)(GDN2_LDS const char*)p; }
template <typename V> __device__ __forceinline__ V lds_get(Lds at) { return *(GDN2_LDS const V*)(uintptr_t)at; }
__device__ __forceinline__ Lds opaque(Lds x) {
    asm volatile("" : "+v"(x));
    return x;
}

// a value that is the same in every lane, in scalar registers
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}

// A buffer resource's words (uniform): loads beyond `bytes` give zeros.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4 rsrc_words(const void* p, uint32_t bytes) {
    const uint64_t a = (uint64_t)(uintptr_t)p;
    return u32x4{(uint32_t)uniform((int)a), (uint32_t)uniform((int)(a >> 32)) & 0xffffu, (uint32_t)uniform((int)bytes), 0x00020000u};
}
// 16 bytes a lane from `off` behind the resource's base to LDS, lane after lane from `to` (uniform) on.
// In assembly because the compiler takes every read of LDS for one of what such a load writes, and
// waits for it; the waits for what arrives are tile_barrier's.  The load has no result registers.  The compiler
// puts no wait states into assembly either: a load reads m0 one state after its write at the earliest, and its
// resource five states after a vector instruction (the readfirstlanes of rsrc_words, a spilled register's
// return) has written a word of it.  The write of m0 and s_nop 3 are five.  (m0 is a clobber, so that the compiler
// takes no value of its own in it for kept; that it never allocates m0 anyway is what the warning would say.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(Lds to, u32x4 r, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(uniform((int)to)), "v"(off), "s"(r)
                 : "memory", "m0");
}

// 16 bytes a lane from each lane's own address (no scalar operand but m0)
__device__ __forceinline__ void load_far_to_lds(Lds to, const void* from) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(uniform((int)to)), "v"(from) : "memory", "m0");
}

// the same, 4 bytes a lane
__device__ __forceinline__ void load_far_words_to_lds(Lds to, const void* from) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(uniform((int)to)), "v"(from) : "memory", "m0");
}
#pragma clang diagnostic pop

// A tile of rows of D elements in LDS, filled by loads that go there directly; it begins at a multiple
// of 1024 bytes.  Rows lie one behind the other without padding (such a load writes 64 lanes' 16-byte
// units in lane order), so each row's units are permuted by an exclusive or.  LDS serves 256 bytes at a
// time: 16 lanes of a row-wise read, which are 16 rows' units, or 32 lanes of a transposing read, which
// are 4 rows' quads of units; either come from different banks.
template <typename T, int D> struct Tile {
    static constexpr int kRow = D * (int)sizeof(T), kUnits = kRow / 16;
    __device__ static constexpr int swz(int row) {
        return (kUnits >= 16 ? (row & 3) << 2 : (row & 2) << 1) | ((row >> 2) & 3);
    }
    // ROWS rows from memory, rows behind `bytes` as zeros; the waves of a workgroup share them
    template <int ROWS, int NW>
    __device__ static __forceinline__ void stage(Lds lds, const void* src, uint32_t bytes, uint32_t stride, int wave,
                                                 int lane) {
        const u32x4 r = rsrc_words(src, bytes);
        constexpr int kLoads = ROWS * kUnits / 64;
        static_assert(ROWS * kUnits % 64 == 0 && kLoads % NW == 0, "whole loads for each wave");
#pragma unroll
        for (int i = 0; i < kLoads / NW; ++i) {
            const int u = (i * NW + wave) * 64 + lane, row = u / kUnits;
            const uint32_t off = (uint32_t)row * stride + (((u % kUnits) ^ swz(row)) << 4);
            load_to_lds(lds + (i * NW + wave) * 1024, r, off);
        }
    }
    // operand of row row0 + l % 32 (row0 a multiple of 16), columns 16 ks + slot in the contiguous map;
    // base: row_base plus the tile's address
    __device__ static __forceinline__ Lds row_base(int lane) {
        const int row = lane & 31, g = lane >> 5;
        return row * kRow + (((sizeof(T) == 2 ? g : 2 * g) ^ swz(row)) << 4);
    }
    __device__ static __forceinline__ Op<T> row_op(Lds base, int row0, int ks) {
        Op<T> r;
        if constexpr (sizeof(T) == 2) {
            r.v = lds_get<bf16x8>((base ^ (ks << 5)) + row0 * kRow);
        } else {
            const f32x4 lo = lds_get<f32x4>((base ^ (ks << 6)) + row0 * kRow);
            const f32x4 hi = lds_get<f32x4>((base ^ (ks << 6) ^ 16) + row0 * kRow);
#pragma unroll
            for (int e = 0; e < 4; ++e) { r.v[e] = lo[e]; r.v[e + 4] = hi[e]; }
        }
        return r;
    }
    // operand of column 32 dt + l % 32, rows row0 + slot (row0 a multiple of 16) in the permuted map;
    // base: col_base plus the tile's address
    __device__ static __forceinline__ Lds col_base(int lane) {
        const int g = lane >> 5;
        if constexpr (sizeof(T) == 2) {
            // a transposing read: 16 lanes give 4 rows of 16 columns and get a column's 4 rows each
            const int j = lane & 15, row = 4 * g + (j >> 2), unit = 2 * ((lane >> 4) & 1) + ((j & 3) >> 1);
            return row * kRow + ((unit ^ swz(row)) << 4) + ((j & 1) << 3);
        } else {
            const int c = lane & 31;
            return 4 * g * kRow + (((c >> 2) ^ swz(4 * g)) << 4) + (c & 3) * 4;
        }
    }
    __device__ static __forceinline__ Op<T> col_op(Lds base, int row0, int dt) {
        Op<T> r;
        if constexpr (sizeof(T) == 2) {
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            bf16x4 h[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                h[k] = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((GDN2_LDS s16x4*)(uintptr_t)(
                                                      (base ^ (4 * dt << 4) ^ (swz(8 * k) << 4)) + (row0 + 8 * k) * kRow)));
            r.v = __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = 8 * (e / 4) + e % 4;
                r.v[e] = lds_get<float>((base ^ (8 * dt << 4) ^ (swz(row) << 4)) + (row0 + row) * kRow);
            }
        }
        return r;
    }
};

// operand of a row in memory, columns 16 ks + slot in the contiguous map; rows behind `bytes` as zeros
template <typename T>
__device__ __forceinline__ Op<T> global_op(__amdgpu_buffer_rsrc_t r, uint32_t row_off, int ks, int g) {
    Op<T> o;
    const uint32_t off = row_off + (16 * ks + 8 * g) * (uint32_t)sizeof(T);
    if constexpr (sizeof(T) == 2) {
        o.v = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
    } else {
        const f32x4 lo = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
        const f32x4 hi = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 16, 0, 0));
#pragma unroll
        for (int e = 0; e < 4; ++e) { o.v[e] = lo[e]; o.v[e + 4] = hi[e]; }
    }
    return o;
}

// bytes from the first of `rows` rows to the end of the last's `width` bytes (0 for none)
__device__ __forceinline__ uint32_t span(int rows, uint32_t stride, uint32_t width) {
    return rows > 0 ? (uint32_t)(rows - 1) * stride + width : 0u;
}

// 4 consecutive columns of each 8 of an accumulator's column: a lane's part of a row of D elements
template <typename T, int D>
__device__ __forceinline__ void store_column(T* row, const f32x16 (&c)[D / 32], float factor, int g) {
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = c[dt][4 * q + e] * factor;
            store_vec_any<T, 4>(row + 32 * dt + 8 * q + 4 * g, f);
        }
}

// The same for a wave's 32 rows (`rows` of them there), through LDS of the wave's own, so that whole rows
// go out 16 bytes a lane instead of 8 bytes of each row.  `to`: the first row's; `stride`: bytes between rows.
template <typename T, int D>
__device__ __forceinline__ void store_rows(Lds lds, char* to, int64_t stride, int rows, const f32x16 (&c)[D / 32], float factor,
                                           int lane) {
    typedef Tile<T, D> L;
    const int row = lane & 31, g = lane >> 5;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int byte = (32 * dt + 8 * q + 4 * g) * (int)sizeof(T);
            const Lds at = lds + row * L::kRow + (((byte >> 4) ^ L::swz(row)) << 4) + (byte & 15);
            if constexpr (sizeof(T) == 2) {
                bf16x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = from_f32<bf16>(c[dt][4 * q + e] * factor);
                *(GDN2_LDS bf16x4*)(uintptr_t)at = v;
            } else {
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = c[dt][4 * q + e] * factor;
                *(GDN2_LDS f32x4*)(uintptr_t)at = v;
            }
        }
    __builtin_amdgcn_wave_barrier();  // a wave's reads of LDS follow its writes in order
#pragma unroll
    for (int i = 0; i < 32 * L::kUnits / 64; ++i) {
        const int u = i * 64 + lane, r = u / L::kUnits, unit = u % L::kUnits;
        const u32x4 v = lds_get<u32x4>(lds + r * L::kRow + ((unit ^ L::swz(r)) << 4));
        if (r < rows) *reinterpret_cast<u32x4*>(to + r * stride + unit * 16) = v;
    }
}

// v of the lane 32 away: the other half of an accumulator's column
__device__ __forceinline__ float other_half(float v, int lane) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, v), __builtin_bit_cast(unsigned, v), false, false);
    return __builtin_bit_cast(float, lane < 32 ? r[1] : r[0]);
}

// every wave is here, and what they wrote to LDS can be read; loads and stores are not waited for
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// loads that go to LDS directly have arrived, and every wave is here
__device__ __forceinline__ void tile_barrier() {
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    __syncthreads();
}

// The same for a wave's own loads and LDS; what it read there has arrived, too.
__device__ __forceinline__ void own_tile_wait() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// Sums over SW waves, in the order of the waves, of the 32 x D that each holds: each wave gets a part of
// them, columns 8 (wave kUnits + u) + 4 g + e of row l % 32.  Takes kBytes of LDS, where nobody reads any
// more; whoever writes there next waits for every wave first.
template <int D, int SW> struct WaveSums {
    static constexpr int kUnits = D / 8 / SW, kBytes = SW * D / 8 * 1024;
    f32x4 v[kUnits];
    __device__ __forceinline__ void add(Lds lds, const f32x16 (&c)[D / 32], float factor, int wave, int lane) {
#pragma unroll
        for (int u = 0; u < D / 8; ++u) {
            f32x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = c[u / 4][4 * (u % 4) + e] * factor;
            *(GDN2_LDS f32x4*)(uintptr_t)(lds + ((wave * (D / 8) + u) * 64 + lane) * 16) = x;
        }
        lds_barrier();
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const Lds at = lds + ((wave * kUnits + u) * 64 + lane) * 16;
            v[u] = lds_get<f32x4>(at);
#pragma unroll
            for (int w = 1; w < SW; ++w) v[u] += lds_get<f32x4>(at + w * (D / 8) * 1024);
        }
    }
    template <typename T> __device__ __forceinline__ void store(T* row, float factor, int wave, int g) const {
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = v[u][e] * factor;
            store_vec_any<T, 4>(row + 8 * (wave * kUnits + u) + 4 * g, f);
        }
    }
};

// zero times x, added to `sum`: a NaN once anything was not finite
__device__ __forceinline__ float watch(float sum, float x) { return __builtin_fmaf(x, 0.f, sum); }

// a value's size as a number that grows with it: that of an infinity is larger than any, that of a NaN larger still
__device__ __forceinline__ unsigned size_bits(float x) { return __builtin_bit_cast(unsigned, x) & 0x7fffffffu; }

// ---- values that are not finite -------------------------------------------------------------
// A product over a tile's rows multiplies what a mask hides by zero, which an infinity or a NaN there
// survives.  Kernels therefore take tiles as they are and look at what came of it; where something is not
// finite, the workgroup starts again in a form in which, in tiles that a mask cuts, a product with the mask
// itself says which infinities and NaN each column sees, and the tile's finite part meets the weights.

__device__ __forceinline__ bool finite_bits(bf16 x) { return (__builtin_bit_cast(unsigned short, x) & 0x7f80u) != 0x7f80u; }
__device__ __forceinline__ bool finite_bits(float x) { return (__builtin_bit_cast(unsigned, x) & 0x7f800000u) != 0x7f800000u; }

template <typename T> __device__ __forceinline__ Op<T> finite_part(Op<T> a) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (!finite_bits((T)a.v[e])) a.v[e] = from_f32<T>(0.f);
    return a;
}
// 1 for a NaN, 128 for an infinity, 16384 for a negative one: sums over up to 64 rows keep the three
// counts apart, and are exact
template <typename T> __device__ __forceinline__ Op<T> special_code(const Op<T>& a) {
    Op<T> r;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float f = to_f32((T)a.v[e]);
        const bool special = !finite_bits((T)a.v[e]);
        r.v[e] = from_f32<T>(!special ? 0.f : f != f ? 1.f : f > 0.f ? 128.f : 16384.f);
    }
    return r;
}
__device__ __forceinline__ float from_code(float c) {
    const float neg = floorf(c * (1.f / 16384.f)), rest = c - neg * 16384.f, pos = floorf(rest * (1.f / 128.f));
    const bool nan = rest - pos * 128.f > 0.f || (neg > 0.f && pos > 0.f);
    return nan ? __builtin_nanf("") : pos > 0.f ? __builtin_inff() : neg > 0.f ? -__builtin_inff() : 0.f;
}

// Which rows of a tile a lane's column has to do with: n of them from lo on.
struct Seen {
    int lo;
    unsigned n;
    __device__ __forceinline__ bool operator()(int row) const { return (unsigned)(row - lo) < n; }
};
__device__ __forceinline__ Seen seen_between(int lo, int hi) { return Seen{lo, hi < lo ? 0u : (unsigned)(hi - lo) + 1u}; }

// What is not finite in column 32 dt + register's row of the tile's rows that a lane's column sees:
// zero, an infinity or a NaN to add (`nan`: a NaN for infinities too, where weights may be zero).
template <typename T, int D, int ROWS>
__device__ __forceinline__ f32x16 special_sum(Lds base, int dt, Seen seen, int g, bool nan) {
    static_assert(ROWS <= 64, "counts below 128");
    f32x16 code = zero16();
#pragma unroll 1
    for (int ks = 0; ks < ROWS / 16; ++ks) {
        Op<T> see;
#pragma unroll
        for (int e = 0; e < 8; ++e) see.v[e] = from_f32<T>(seen(16 * ks + acc_row(e, g)) ? 1.f : 0.f);
        mma(code, special_code<T>(Tile<T, D>::col_op(base, 16 * ks, dt)), see);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) code[i] = nan && code[i] > 0.f ? __builtin_nanf("") : from_code(code[i]);
    return code;
}
// ---- which workgroup does what --------------------------------------------------------------

struct Seq {
    int64_t q0, k0;  // first token of the sequence's queries and keys
    int lq, lk;      // how many there are
};
__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

// Blocks of `rows` tokens of the packed sequences, counted through: sequence and block of the `index`th one,
// or false behind the last.  Up to 64 sequences are counted from the longest to the shortest, so that long ones
// do not start late.  Every wave looks for itself, 64 sequences at a time.
__device__ __forceinline__ bool find_block(const int64_t* cu, int64_t n, int64_t total, int rows, unsigned index, int lane,
                                           int64_t* seq, int* block, int* blocks) {
    int64_t before = 0;
    for (int64_t base = 0; base < n; base += 64) {
        int mine = 0;
        if (base + lane < n) {
            const int64_t lo = clamp64(cu[base + lane], 0, total), hi = clamp64(cu[base + lane + 1], lo, total);
            mine = (int)((hi - lo + rows - 1) / rows);
        }
        int64_t first = before;  // blocks before the lane's
        if (n <= 64) {
            for (int j = 0; j < (int)n; ++j) {
                const int other = __builtin_amdgcn_readlane(mine, j);
                first += other > mine || (other == mine && j < lane) ? other : 0;
            }
        } else {
            int64_t sum = mine;
#pragma unroll
            for (int s = 1; s < 64; s *= 2) {
                const int64_t up = __shfl_up(sum, s);
                if (lane >= s) sum += up;
            }
            first += sum - mine;
            before += __shfl(sum, 63);
        }
        const uint64_t here = __ballot(first <= index && index < first + mine);
        if (here) {
            const int at = __builtin_ctzll(here);
            *seq = base + at;
            *block = (int)(index - __shfl(first, at));
            *blocks = __shfl(mine, at);
            return true;
        }
    }
    return false;
}
__device__ __forceinline__ Seq packed_seq(const int64_t* cu_q, const int64_t* cu_k, int64_t n, int64_t total_q, int64_t total_k) {
    Seq s;
    s.q0 = clamp64(cu_q[n], 0, total_q);
    s.lq = (int)(clamp64(cu_q[n + 1], s.q0, total_q) - s.q0);
    s.k0 = clamp64(cu_k[n], 0, total_k);
    s.lk = (int)(clamp64(cu_k[n + 1], s.k0, total_k) - s.k0);
    return s;
}

// What every attention kernel takes.
struct Shape {
    const int64_t* cu_q;  // packed sequences' offsets, or nullptr
    const int64_t* cu_k;
    int64_t n, tq, tk;    // sequences; tokens of each, or of all packed ones
    int heads, groups, window;
    uint32_t q_stride, k_stride, v_stride;  // bytes between tokens
    float scale, scale_log2;                // scale, and scale log2(e)
    int blocks;           // blocks of a head: of every sequence's, or of all packed ones
    unsigned all_groups;  // key heads of all sequences (packed: key heads)
    int slice_bits;       // a group's blocks are dealt out in 2^slice_bits slices, so that every XCD has as many
    unsigned turn;        // slices of an XCD that take turns
};

// Workgroups go to the 8 XCDs in turn, each with an L2 of its own: the blocks of one group (a
// sequence's key head; packed, a key head) stay on one XCD, or with fewer groups than XCDs are dealt
// out in `slices`.  Within a slice the blocks with the most work come first, the heads of the group
// side by side.  `turn` slices of an XCD take turns, so that no heavy block starts late: as many as make kTurn
// workgroups, and no more, because those that run at once share keys and values in L2.  Forward and backward
// pass, us, one slice after the other, with 256 and with 8192 workgroups: 8 x 1024 tokens of 16 heads of 128, 63,
// 50, 50 and 203, 172, 173; 32 x 4096 tokens, 2296, 2308, 3684 and 7347, 7089, 8926; the gradients of 16 packed
// sequences of 20 to 4096 tokens, 12 heads of 64, 249 and 196 with 256.
struct Work {
    Seq s;
    int block, head;  // head: of `per_group` in each group
};
__device__ __forceinline__ bool find_work(const Shape& p, int rows, int per_group, bool last_first, bool keys, int lane, Work* w) {
    const unsigned x = blockIdx.x & 7, r = blockIdx.x >> 3;
    const unsigned per = (p.blocks + (1u << p.slice_bits) - 1) >> p.slice_bits, each = per * per_group;
    const unsigned slices = ((p.all_groups << p.slice_bits) + 7) >> 3, before = r / (each * p.turn) * p.turn;  // of an XCD
    const unsigned width = min(slices - before, p.turn), rest = r % (each * p.turn) / (unsigned)per_group;
    const unsigned slice = (before + rest % width) * 8 + x, group = slice >> p.slice_bits, nth = rest / width;
    // A group's slices go round with its number: with fewer blocks than slices the last ones are empty, and would
    // be the same XCDs' for every group (9 x 351 tokens, 16 heads of 128 sharing one, fp32: dq 320 us, 137 so).
    const unsigned of_group = (slice + (slice >> 3)) & ((1u << p.slice_bits) - 1);
    const unsigned index = ((last_first && !p.cu_q ? per - 1 - nth : nth) << p.slice_bits) + of_group;
    if (group >= p.all_groups || index >= (unsigned)p.blocks) return false;
    w->head = (int)(group % (unsigned)p.groups) * per_group + r % (unsigned)per_group;
    if (p.cu_q) {
        int64_t seq;
        int blocks;
        if (!find_block(keys ? p.cu_k : p.cu_q, p.n, keys ? p.tk : p.tq, rows, index, lane, &seq, &w->block, &blocks)) return false;
        if (last_first) w->block = blocks - 1 - w->block;
        w->s = packed_seq(p.cu_q, p.cu_k, seq, p.tq, p.tk);
    } else {
        const int64_t n = group / (unsigned)p.groups;
        w->s = Seq{n * p.tq, n * p.tk, (int)p.tq, (int)p.tk};
        w->block = (int)index;
    }
    return true;
}
// the same in every lane: in scalar registers
__device__ __forceinline__ Work uniform(const Work& w) {
    return Work{Seq{uniform(w.s.q0), uniform(w.s.k0), uniform(w.s.lq), uniform(w.s.lk)}, uniform(w.block), uniform(w.head)};
}
constexpr int64_t kTurn = 256;
constexpr int64_t kMaxWork = (int64_t)1 << 23;  // blocks of all heads
constexpr int64_t kMaxGrid = (int64_t)1 << 24;  // workgroups of 256 threads: a launch has less than 2^32
// Fills in how work is dealt out; workgroups of the launch (0: none), or -1 if there is too much work.  Slices without
// a block, and groups that are missing to a multiple of the XCDs, make the launch larger than the work.  So many
// groups of few blocks are cut into no more slices than they have blocks (1025 sequences of 60 tokens, 4 heads of 64
// sharing one: 53 us with 8 slices, 30 with one, the gradients 135 and 72), and slices are fewer where the launch
// would not fit.  Then it does: 8 blocks or more are less than doubled by any slices, and 2^20 heads of fewer are 16
// groups or more, which are less than doubled without.
inline int64_t deal(Shape* p, int64_t tokens, int rows, int per_group) {
    const int64_t blocks = p->cu_q ? tokens / rows + p->n : (tokens + rows - 1) / rows;
    const int64_t groups = p->cu_q ? p->groups : p->n * p->groups;
    if (blocks == 0) return 0;
    if (blocks >= kMaxWork || groups >= kMaxWork || blocks * groups >= kMaxWork || blocks * groups * per_group >= kMaxWork) return -1;
    p->blocks = (int)blocks;
    p->all_groups = (unsigned)groups;
    auto per = [&] { return (blocks + ((int64_t)1 << p->slice_bits) - 1) >> p->slice_bits; };
    auto slices = [&] { return ((groups << p->slice_bits) + 7) / 8; };  // of an XCD
    auto grid = [&] { return slices() * 8 * per() * per_group; };
    p->slice_bits = 0;
    while ((groups << p->slice_bits) % 8 && (groups < 64 || (2 << p->slice_bits) <= blocks)) ++p->slice_bits;
    while (p->slice_bits > 0 && grid() >= kMaxGrid) --p->slice_bits;
    p->turn = (unsigned)min(slices(), (kTurn + per() * per_group - 1) / (per() * per_group));
    return grid() < kMaxGrid ? grid() : -1;
}

// Rows whose keys were taken in parts: unnormalised sums o [splits][rows][d] in fp32, and of each row
// and part the reference (base 2) and the sum (ml).  lse may be nullptr.
struct Parts {
    float* o;
    float2* ml;
    int64_t rows;
    int splits;
};
inline size_t parts_bytes(int64_t rows, int64_t d, int splits) { return (size_t)splits * (size_t)rows * (size_t)(d + 2) * 4; }
inline Parts parts_in(void* workspace, int64_t rows, int64_t d, int splits) {
    float* o = static_cast<float*>(workspace);
    return Parts{o, reinterpret_cast<float2*>(o + splits * rows * d), rows, splits};
}
// the tokens that rows belong to, `heads` rows each: all (no offsets), or those of packed sequences
struct Owned {
    const int64_t* cu;
    int64_t n, total;
    int heads;
};
// whether a token belongs to a sequence; each lane asks for its own
__device__ __forceinline__ bool owned_by_lane(const Owned& o, int64_t token) {
    if (!o.cu) return true;
    bool found = false;
    for (int64_t n = 0; n < o.n && !found; ++n) {
        const int64_t lo = clamp64(o.cu[n], 0, o.total);
        found = lo <= token && token < clamp64(o.cu[n + 1], lo, o.total);
    }
    return found;
}
hipError_t launch_join(const Parts& p, void* o, float* lse, int64_t d, bool bf16_out, const Owned& owned, hipStream_t stream);

}  // namespace attn
}  // namespace gdn2
