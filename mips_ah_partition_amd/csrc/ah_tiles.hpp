// Matrix products of a learned query side on the CDNA4 matrix cores: the tiled contraction and
// the one for few rows, which ah_products.hip, ah_gated.hip and ah_f8.hip instantiate for their operands.
//
// All of them are one contraction, out[i][j] = sum_t Q[i][t] P[j][t], with Q the
// row side (tokens) and P the column side (channels):
//   int8     Q = codes [m][k],           P = codes [n][k]            t = k
//   forward  Q = queries of a leaf,      P = the leaf's W [n][k]     t = k
//   dx       Q = slot gradients,         P = the leaf's W, by column t = n
//   dw       Q = slot gradients by column, P = queries by column     t = the leaf's rows
//   gate     Q = queries of a leaf,      P = the leaf's gate and up rows [2n][k], in turn: a wave has both of a column
//   grad     as dx, of a gated block's output layer
//   float8   Q = codes [m][kp],          P = codes [n][kp]           t = kp, a scale for each row and step
// "By column" operands have the summed index along memory rows; their LDS tiles
// are read with the transposing LDS load (ds_read_b64_tr_b16).
//
// Tiles.  One step of the sum is 128 bytes of t (128 int8 or 64 bfloat16 values), and
// every operand's step is cut into blocks of 8 KB: 64 rows x 128 bytes ("row" operands)
// or 64 memory rows x 64 columns ("by column").  Global memory goes straight to LDS (16
// bytes a lane); that write is linear in the lane, so the swizzle that keeps the reads
// free of bank conflicts is applied to the source address.  A row operand's 16-byte
// chunk c of row r lies at c ^ key(r).  A 16-byte read serves lanes 0-3, 12-15, 20-23 and 24-27 at
// once (then 4-11, 16-19, 28-31, and the upper half alike), so key has to tell apart rows 0-3 from
// 12-15 and 4-7 from 8-11 of a fragment read in order, and the same of rows 8 a + b (PERM):
// r & 3 with the parity of bits 2 and 4 above it does (0 conflicts counted; r & 7, without
// PERM, too).  A by-column operand's 32-byte granule c of memory row r lies at c ^ (r >> 1 & 1 | (r >> 3
// & 1) << 1).  The matrix instruction takes P as its A operand, so
// that a lane ends with four consecutive output columns of one row.
#pragma once
#include <type_traits>

#include "ah_device.hpp"
#include "ah_gating.hpp"
#include "ah_kernels.hpp"
#include "../../include/ah.h"

namespace ah {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

enum { kI8 = 0, kFwd = 1, kDx = 2, kDw = 3, kGate = 4, kGrad = 5, kF8 = 8 };  // kF8 + Q's type + 2 * P's type
constexpr bool is_f8(int mode) { return mode >= kF8; }
constexpr bool is_plain(int mode) { return mode == kI8 || is_f8(mode); }  // one matrix, rows in order
constexpr bool is_gated(int mode) { return mode == kGate || mode == kGrad; }
constexpr bool is_ragged(int mode) { return !is_plain(mode) && mode != kDw; }
constexpr bool p_by_col(int mode) { return mode == kDx || mode == kDw || mode == kGrad; }
constexpr int elem_bytes(int mode) { return is_plain(mode) ? 1 : 2; }

constexpr int kNT = 256;     // threads: 2 x 2 waves
constexpr int kCUs = 256;    // compute units of an MI355X (a multiple of its 8 XCDs)
constexpr int kBlock = 8192; // bytes of a block

// Source of chunks that lie outside an operand (past its sum or its columns).
__device__ const v4i zero_chunk = {0, 0, 0, 0};
// Source of a whole step past the sum, for float8 operands whose rows are one step long: 256 rows of 128 bytes.
__device__ const v4i zero_rows[2048] = {};

struct ProdArgs {
    const char* q;         // row side
    const char* p;         // column side
    int64_t qs, ps;        // bytes between memory rows
    int64_t pg;            // bytes between the leaves' matrices (forward, dx)
    const int64_t* off;    // leaf starts [L + 1]
    const int32_t* order;  // slot of each grouped row, or NULL: the row itself
    int64_t T;             // grouped rows (int8: m)
    int32_t L;
    uint32_t fan_mul, fan_shift;  // s / fan = s * fan_mul >> fan_shift
    int64_t I, J;          // output rows of one matrix (dw: n; else T) and columns
    int64_t red;           // summed elements (dw: unused, the leaf's rows)
    void* out;
    int32_t out_f32;
    int32_t bypass;        // rows of whole 64-byte sectors (gated products have stores of their own)
    const float *sx, *sw, *bias;  // int8 (bias: float8 too)
    int32_t act;           // gated: activation, dropout, the projections [slots][2 J] (gate: written, or NULL; grad: read)
    Dropout drop;          // and h (grad; or NULL)
    char *pre, *hidden;
    const char *qsc, *psc; // float8: scale bytes [steps][pitch]
    int64_t qpitch, ppitch;
};

typedef const __attribute__((address_space(3))) v4i* lds_v4i;
typedef __attribute__((address_space(3))) v4s* lds_v4s;
typedef __attribute__((address_space(3))) char* lds_char;

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}
// 16 bytes a lane from global memory to LDS, at lds + 16 * lane.  Written out because for the
// builtin the compiler lets every later LDS read wait for all loads in flight, which
// would undo the prefetch; the loops below wait by themselves (land).  It has no
// output registers, so nothing that the compiler allocates can be overwritten by it, and
// m0, which the compiler keeps nothing in, is set in the same block.
__device__ __forceinline__ void dma16(const char* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(
                     __builtin_amdgcn_readfirstlane(lds)),
                 "v"(src));
}
// The same from a uniform address and an offset a lane, to a uniform one.
__device__ __forceinline__ void dma16(const char* src, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(src));
}
// 4 bytes a lane, at lds + 4 * lane.
__device__ __forceinline__ void dma4(const char* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(
                     __builtin_amdgcn_readfirstlane(lds)),
                 "v"(src));
}
// Barrier at which all but the newest N of a wave's memory operations have landed and its LDS
// reads are done.  (The builtin wait, unlike one in asm, is seen by the compiler: it
// places no waits of its own for loads that were started before.)
template <int N>
__device__ __forceinline__ void land() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 7 << 4);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

template <int MODE>
struct Acc {
    typedef v4f type;
};
template <>
struct Acc<kI8> {
    typedef v4i type;
};
template <int MODE>
__device__ __forceinline__ typename Acc<MODE>::type mma(v4i p, v4i q, typename Acc<MODE>::type c) {
    if constexpr (MODE == kI8)
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(p, q, c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, p), __builtin_bit_cast(v8bf, q), c, 0,
                                                       0, 0);
}

// 128 bytes of the sum; scale bytes in the low bytes of sp and sq.
__device__ __forceinline__ v8i halves(v4i lo, v4i hi) {
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <int MODE>
__device__ __forceinline__ v4f mma8(v8i p, v8i q, v4f c, int sp, int sq) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, c, (MODE - kF8) >> 1 & 1, (MODE - kF8) & 1, 0, sp, 0,
                                                            sq);
}

// Element of an accumulator that is kept in the accumulation registers.  (All its uses but the
// matrix instruction are written like this and held(): left to itself the compiler keeps the sums
// in vector registers and moves each in and out of the accumulation registers, 8 moves an
// instruction.)  Before the first read after matrix instructions: settle().
template <typename T>
__device__ __forceinline__ T acc_read(T c) {
    T v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(c));
    return v;
}
template <typename T>
__device__ __forceinline__ void held(T& c) {
    asm volatile("" : "+a"(c));
}
// The wait states between a matrix instruction and a read of its result; for acc_read, which the
// compiler does not look into, they have to be written down.
__device__ __forceinline__ void settle() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 7");
    __builtin_amdgcn_sched_barrier(0);
}

// The 16 bytes v moved down by `cut` bytes (< 16), zeros above.
__device__ __forceinline__ v4i shift_down(v4i v, int cut) {
    const uint64_t lo = (uint32_t)v[0] | (uint64_t)(uint32_t)v[1] << 32,
                   hi = (uint32_t)v[2] | (uint64_t)(uint32_t)v[3] << 32;
    const int n = 8 * (cut & 7);
    const uint64_t a = cut & 8 ? hi : lo, b = cut & 8 ? 0 : hi;
    const uint64_t l = a >> n | (b << 1) << (63 - n), h = b >> n;
    return v4i{(int)(uint32_t)l, (int)(uint32_t)(l >> 32), (int)(uint32_t)h, (int)(uint32_t)(h >> 32)};
}
// 16 bytes of a row of which the first `valid` exist (<= 0: none), `before` bytes into the row; ELEM
// bytes an element.  A row's short end is read as the 16 bytes up to it, moved down; element by
// element only in rows of less than 16 bytes.
template <int ELEM>
__device__ __forceinline__ v4i load_chunk(const char* src, int64_t valid, int64_t before) {
    v4i r = {0, 0, 0, 0};
    if (valid <= 0) return r;
    const int cut = valid >= 16 ? 0 : 16 - (int)valid;
    if (before >= cut) {
        __builtin_memcpy(&r, src - cut, 16);
        if (cut > 0) r = shift_down(r, cut);
    } else {
        for (int b = 0; b < (int)valid; b += ELEM) {  // the last element comes down to the bottom
            uint32_t e = 0;
            __builtin_memcpy(&e, src + (int)valid - ELEM - b, ELEM);
            uint64_t lo = (uint32_t)r[0] | (uint64_t)(uint32_t)r[1] << 32, hi = (uint32_t)r[2] | (uint64_t)(uint32_t)r[3] << 32;
            hi = hi << (8 * ELEM) | lo >> (64 - 8 * ELEM);
            lo = lo << (8 * ELEM) | e;
            r = v4i{(int)(uint32_t)lo, (int)(uint32_t)(lo >> 32), (int)(uint32_t)hi, (int)(uint32_t)(hi >> 32)};
        }
    }
    return r;
}

__device__ __forceinline__ uint32_t bf16_bits(float f) {  // round to nearest even; NaN stays NaN
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f);
}
// Two of them, in one instruction where the scalar ones take two and three to join them.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}
// One wave's 32 NQ x 32 NP results to memory; sc holds the int8 scales of the tile (its 64 NP columns'
// scales, their biases, its 64 NQ rows' steps).  The matrix instruction leaves four columns of a
// row in a lane, 16 rows in a wave.
//   bfloat16  the column side's fragments are read so that two of them give a lane eight
//             consecutive columns (PERM; not by column): a store is 16 rows x 64 bytes
//   float32   16 rows at a time, all columns (NP = 2: half of them), are turned around in LDS, rows
//             16 bytes further apart than they are long, and stored in that order (two conflicts an
//             access by the counters, of about 128 accesses a tile and wave; operand reads have none)
// Where rows are made of whole 64-byte sectors the stores bypass the caches' reuse order: the
// results are not read here, and kept as others they push operands out of L2 (int8 to bfloat16,
// 8192 x 4096 x 16384: 600 us without, 529 with).  Rows at other pitches share sectors and are
// merged in L2 (float32, 1000 x 1536 x 100003: 424 us bypassing, 270 not).

// A value that the compiler takes as new at this place: what is computed from it is not moved out of the
// loop over tiles, where it would hold registers that the matrix loop needs.
__device__ __forceinline__ int here(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

template <int MODE, int OB>
constexpr bool kPerm = OB == 2 && !p_by_col(MODE);
template <int NP>
constexpr int kTurnCols = NP == 4 ? 64 : 32;
template <int NP>
constexpr int kTurnPitch = kTurnCols<NP> * 4 + 16;

// The first `left` (0 < left < n) of n elements of OB bytes, in pieces of 8, 4 and 2 bytes: element by element
// the epilogues' code would outgrow the instruction cache.
template <int OB>
__device__ __forceinline__ void store_left(char* o, v4i v, int32_t left) {
    const int32_t bytes = left * OB;
    const bool up = bytes & 8;
    if (up) __builtin_memcpy(o, &v, 8);
    const int a = up ? v[2] : v[0], b = up ? v[3] : v[1];
    o += bytes & 8;
    if (bytes & 4) __builtin_memcpy(o, &a, 4);
    if constexpr (OB == 2) {
        const uint16_t c = (uint16_t)(bytes & 4 ? b : a);
        if (bytes & 2) __builtin_memcpy(o + (bytes & 4), &c, 2);
    }
}
__device__ __forceinline__ void store16(char* o, v4i v, int32_t bypass) {
    if (bypass)
        __builtin_nontemporal_store(v, reinterpret_cast<v4i*>(o));
    else
        __builtin_memcpy(o, &v, 16);
}

template <int MODE, int NQ, int NP, int OB>
__device__ __forceinline__ void store_part(const ProdArgs& a, typename Acc<MODE>::type (&acc)[2 * NQ][2 * NP],
                                           const float* sc, char* turn, const int32_t (&out_row)[2], int32_t leaf,
                                           int32_t j0) {
    constexpr int FQ = 2 * NQ, FP = 2 * NP, Y = kPerm<MODE, OB> ? 2 : 1;  // fragments behind a lane's run of columns
    constexpr int N = 4 * Y;                                             // columns of that run
    const int tid = here(threadIdx.x), lane = tid & 63, wave = tid >> 6, g = lane >> 4, li = lane & 15;
    const int wq = wave >> 1, wp = wave & 1;
    const int c0 = wp * 32 * NP;  // the wave's first column in the tile
    const int64_t first = MODE == kDw ? leaf * a.I : 0;
    auto value = [&](int x, int y, float sx, float* v) {
        typename Acc<MODE>::type r = acc[x][y];
        if constexpr (NQ * NP > 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] = acc_read(acc[x][y][e]);
        }
        if constexpr (MODE == kI8) {
            const int c = c0 + (Y == 2 ? (y >> 1) * 32 + g * 8 + (y & 1) * 4 : y * 16 + g * 4);
            const v4f sw = *reinterpret_cast<const v4f*>(sc + c);
            const v4f bias = *reinterpret_cast<const v4f*>(sc + 64 * NP + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = (float)r[e] * sx * sw[e];
                if (a.bias) v[e] += bias[e];
            }
        } else if constexpr (is_f8(MODE)) {
            const v4f bias = *reinterpret_cast<const v4f*>(
                sc + c0 + (Y == 2 ? (y >> 1) * 32 + g * 8 + (y & 1) * 4 : y * 16 + g * 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = r[e] + bias[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = r[e];
        }
    };
    if constexpr (OB == 2) {
        const bool whole = j0 + 64 * NP <= a.J;
#pragma unroll
        for (int x = 0; x < FQ; ++x) {
            const int32_t row = __shfl(out_row[x / 4], (x & 3) * 16 + li, 64);
            float sx = 0.0f;
            if constexpr (MODE == kI8) sx = sc[128 * NP + wq * 32 * NQ + x * 16 + li];
            char* const o = static_cast<char*>(a.out) + ((first + row) * a.J + j0 + c0 + g * N) * 2;
#pragma unroll
            for (int y = 0; y < FP; y += Y) {
                float v[N];
#pragma unroll
                for (int u = 0; u < Y; ++u) value(x, y + u, sx, v + 4 * u);
                uint32_t w[N / 2];
#pragma unroll
                for (int e = 0; e < N / 2; ++e) w[e] = bf16_pair(v[2 * e], v[2 * e + 1]);
                const int32_t left = whole ? N : (int32_t)a.J - (j0 + c0 + g * N + y * 16);
                if (row < 0) {
                } else if (left >= N) {
                    if constexpr (N == 8)
                        store16(o + y * 32, v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]}, a.bypass);
                    else
                        __builtin_memcpy(o + y * 32, w, 8);
                } else if (left > 0) {
                    store_left<2>(o + y * 32, v4i{(int)w[0], (int)w[1], N == 8 ? (int)w[N / 2 - 2] : 0,
                                                  N == 8 ? (int)w[N / 2 - 1] : 0}, left);
                }
                __builtin_amdgcn_sched_barrier(0);  // one store's registers at a time
            }
        }
    } else {
        constexpr int TC = kTurnCols<NP>, PITCH = kTurnPitch<NP>, NC = TC / 4, YP = TC / 16;
#pragma unroll
        for (int x = 0; x < FQ; ++x) {
            float sx = 0.0f;
            if constexpr (MODE == kI8) sx = sc[128 * NP + wq * 32 * NQ + x * 16 + li];
#pragma unroll
            for (int ps = 0; ps < FP / YP; ++ps) {
#pragma unroll
                for (int yy = 0; yy < YP; ++yy) {
                    float e[4];
                    value(x, ps * YP + yy, sx, e);
                    *reinterpret_cast<v4f*>(turn + li * PITCH + (yy * 4 + g) * 16) = v4f{e[0], e[1], e[2], e[3]};
                }
                __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int n = 0; n < NC / 4; ++n) {
                    const int id = n * 64 + lane, r = id / NC, c = id % NC;
                    const int32_t row = __shfl(out_row[x / 4], (x & 3) * 16 + r, 64), j = j0 + c0 + ps * TC + c * 4;
                    const v4i v = *reinterpret_cast<const v4i*>(turn + r * PITCH + c * 16);
                    char* const o = static_cast<char*>(a.out) + ((first + row) * a.J + j) * 4;
                    if (row < 0) {
                    } else if (j + 4 <= a.J) {
                        store16(o, v, a.bypass);
                    } else if (j < a.J) {
                        store_left<4>(o, v, (int32_t)a.J - j);
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
        }
    }
}

// Four consecutive bfloat16 values, of which `left` exist.
__device__ __forceinline__ void put_bf16(char* o, const float* v, int32_t left) {
    const uint32_t w[2] = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    if (left >= 4)
        __builtin_memcpy(o, w, 8);
    else if (left > 0)
        store_left<2>(o, v4i{(int)w[0], (int)w[1], 0, 0}, left);
}
// Eight, as they lie in memory (zeros for those that do not exist).
__device__ __forceinline__ v4i get_bf16x8(const char* p, int32_t left) {
    v4i r = {0, 0, 0, 0};
    if (left >= 8) {
        __builtin_memcpy(&r, p, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint16_t b = 0;
            if (e < left) __builtin_memcpy(&b, p + 2 * e, 2);
            r[e >> 1] |= (int)((uint32_t)b << (e & 1 ? 16 : 0));
        }
    }
    return r;
}
__device__ __forceinline__ float bf16_at(v4i r, int e) {
    return __uint_as_float(e & 1 ? (uint32_t)r[e >> 1] & 0xFFFF0000u : (uint32_t)r[e >> 1] << 16);
}
// Factors of four columns from j on (a multiple of 4) of a row.
__device__ __forceinline__ void dropout_factors(const Dropout& d, uint64_t step, int32_t row, int32_t j, float* f) {
    if (d.t == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = 1.0f;
        return;
    }
    const Philox u = philox(d, step, (uint32_t)row, (uint32_t)j >> 3);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t n = j & 4 ? u.at(e + 4) : u.at(e);
        f[e] = n >= d.t ? d.factor : 0.0f;
    }
}
// A dropped element is 0 whatever it was.
__device__ __forceinline__ float dropped(float v, float f) { return f > 0.0f ? v * f : 0.0f; }

// Which of eight columns from j on (a multiple of 4; the second four are not asked for where it is none of 8) stay, as
// 16-bit masks: u >= t where t - u, not below 0, is 0.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void keep_masks(const Dropout& d, uint64_t step, int32_t row, int32_t j, uint32_t* m) {
    if (d.t == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) m[q] = 0xFFFFFFFFu;
        return;
    }
    const Philox u = philox(d, step, (uint32_t)row, (uint32_t)j >> 3);
    const u16x2 t = {(unsigned short)d.t, (unsigned short)d.t}, one = {1, 1};
#pragma unroll
    for (int q = 0; q < 4; ++q)
        m[q] = __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_elementwise_sub_sat(
                                                t, __builtin_bit_cast(u16x2, u.w[q])), one) - one);
    if (j & 4) {
        m[0] = m[2];
        m[1] = m[3];
    }
}
// N values as bfloat16 under their masks, of which `left` exist.
template <int N>
__device__ __forceinline__ void put_masked(char* o, const float* v, const uint32_t* m, int32_t left) {
    uint32_t w[4] = {};
#pragma unroll
    for (int e = 0; e < N / 2; ++e) w[e] = bf16_pair(v[2 * e], v[2 * e + 1]) & m[e];
    if (left >= N)
        __builtin_memcpy(o, w, 2 * N);
    else if (left > 0)
        store_left<2>(o, v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]}, left);
}
// Fragment row x of the sums.  A switch over a run-time x, so that what follows stands in the code once and not for every
// x: unrolled the gated epilogues would outgrow the instruction cache.
template <int FQ, int FP>
__device__ __forceinline__ void take_row(v4f (&acc)[FQ][FP], int x, v4f (&t)[FP]) {
#pragma unroll
    for (int n = 0; n < FQ; ++n)
        if (x == n) {
#pragma unroll
            for (int i = 0; i < FP * 4; ++i) {
                if constexpr (FQ * FP > 16)
                    t[i >> 2][i & 3] = acc_read(acc[n][i >> 2][i & 3]);
                else
                    asm volatile("v_mov_b32 %0, %1" : "=v"(t[i >> 2][i & 3]) : "v"(acc[n][i >> 2][i & 3]));
            }
        }
}

// Gated product, 16,384 rows of 16 leaves, 1536 -> 2 x 4096 (412 GFLOP), dropout, both projections kept: 538-558 us at 4 x 4.
// The contraction takes 380 of them (without its loads 285; a dense library product of the size 380); what no matrix
// instruction covers are the stores (402 MB, all CUs at once: 77, 5.2 TB/s), the activation and its rounding (60) and Philox
// (46).  Matrix instructions run in 0.36 of the clocks, at 2.0 GHz.
// A wave's part of a gated product: a lane holds gate and up of the same columns, in fragments NP apart.  The
// activation is a template's, chosen once a tile: chosen for each element the compiler computes all and selects.  WHOLE:
// all the tile's columns exist, so that nothing but the rows is asked about.
template <int ACT, bool WHOLE, int NQ, int NP, int OB>
__device__ __forceinline__ void store_gate(const ProdArgs& a, v4f (&acc)[2 * NQ][2 * NP], const int32_t (&out_row)[2],
                                           int32_t j0, uint64_t step) {
    constexpr int FQ = 2 * NQ, Y = OB == 2 ? 2 : 1, N = 4 * Y;
    const int tid = here(threadIdx.x), lane = tid & 63, wave = tid >> 6, g = lane >> 4, li = lane & 15;
    const int32_t jw = j0 + (wave & 1) * 16 * NP + g * N;
    const uint32_t all[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
#pragma nounroll
    for (int x = 0; x < FQ; ++x) {
        const int32_t row = __shfl(x < 4 ? out_row[0] : out_row[1], (x & 3) * 16 + li, 64);
        v4f t[2 * NP];
        take_row(acc, x, t);
        char* const out = static_cast<char*>(a.out) + ((int64_t)row * a.J + jw) * OB;
        char* const pre = a.pre + ((int64_t)row * 2 * a.J + jw) * 2;
        char* const pre_up = pre + a.J * 2;
#pragma unroll
        for (int y = 0; y < NP; y += Y) {
            const int32_t j = jw + y * 16, left = WHOLE ? N : (int32_t)a.J - j;
            float u[N], v[N], h[N];
            uint32_t m[4];
            keep_masks(a.drop, step, row, j, m);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                u[e] = t[y + e / 4][e & 3];
                v[e] = t[y + NP + e / 4][e & 3];
                h[e] = activate(ACT, u[e]) * v[e] * a.drop.factor;
            }
            if (row >= 0 && left > 0) {
                if constexpr (OB == 2) {
                    put_masked<N>(out + y * 32, h, m, left);
                } else {
                    v4i w;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = m[e >> 1] >> (e & 1 ? 16 : 0) & 1 ? __builtin_bit_cast(int, h[e]) : 0;
                    if (left >= 4)
                        __builtin_memcpy(out + y * 64, &w, 16);
                    else
                        store_left<4>(out + y * 64, w, left);
                }
                if (a.pre) {
                    put_masked<N>(pre + y * 32, u, all, left);
                    put_masked<N>(pre_up + y * 32, v, all, left);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// Two column fragments, a lane holding columns 4 g .. 4 g + 3 of each, become eight consecutive columns: with quarters
// of a wave g = 0 .. 3, those of fragment g & 1 from 8 (g >> 1) on.
__device__ __forceinline__ void eight_columns(v4f f0, v4f f1, float* v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(f0[e]), __float_as_uint(f1[e]), false, false);
        v[e] = __uint_as_float(t[0]);
        v[4 + e] = __uint_as_float(t[1]);
    }
}
// Gated gradient, 16,384 rows of 16 leaves, 1536 -> 4096 (206 GFLOP, 922 MB), dropout, hidden values too: 369-379 us at 3 x 4,
// the contraction 172 of them (without its loads 140), stores 80 (402 MB), the reads of the projections 35, Philox 27, the
// rest is the activation, its derivative and their rounding: one after another on every CU, matrix instructions in 0.25 of
// the clocks.  4 x 4 would not leave registers for a fragment row's projections on their way.
// A wave's part of the gradient: dh becomes (da, db) and h.  The projections of fragment row x + 1 are asked for before
// row x is dealt with; where the tile is WHOLE without a branch (rows that are not written read row 0), behind which the
// compiler would wait for all of them.
template <int ACT, bool WHOLE, int NQ, int NP>
__device__ __forceinline__ void store_grad(const ProdArgs& a, v4f (&acc)[2 * NQ][2 * NP], const int32_t (&out_row)[2],
                                           int32_t leaf, int32_t j0, uint64_t step) {
    constexpr int FQ = 2 * NQ, N = 8;
    const int tid = here(threadIdx.x), lane = tid & 63, wave = tid >> 6, g = lane >> 4, li = lane & 15;
    const int32_t jw = j0 + (wave & 1) * 32 * NP + (g & 1) * 16 + (g >> 1) * 8;
    v4i u1[NP], v1[NP];
    int32_t row1;
    auto ask = [&](int x) {
        row1 = __shfl(x < 4 ? out_row[0] : out_row[1], (x & 3) * 16 + li, 64);
        const char* const p = a.pre + ((int64_t)(row1 < 0 ? 0 : row1) * 2 * a.J + jw) * 2;
#pragma unroll
        for (int z = 0; z < NP; ++z) {
            const int32_t left = WHOLE ? N : row1 < 0 ? 0 : (int32_t)a.J - (jw + z * 32);
            u1[z] = get_bf16x8(p + z * 64, left);
            v1[z] = get_bf16x8(p + z * 64 + a.J * 2, left);
        }
    };
    ask(0);
#pragma nounroll
    for (int x = 0; x < FQ; ++x) {
        const int32_t row = row1;
        v4i u[NP], v[NP];
#pragma unroll
        for (int z = 0; z < NP; ++z) {
            u[z] = u1[z];
            v[z] = v1[z];
        }
        if (x + 1 < FQ) ask(x + 1);
        v4f t[2 * NP];
        take_row(acc, x, t);
        char* const gate = static_cast<char*>(a.out) + ((int64_t)row * 2 * a.J + jw) * 2;
        char* const up_to = gate + a.J * 2;
        char* const hidden = a.hidden + ((int64_t)row * a.J + jw) * 2;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int z = 0; z < NP; ++z) {
            const int32_t j = jw + z * 32, left = row < 0 ? 0 : WHOLE ? N : (int32_t)a.J - j;
            float dh[N], da[N], db[N], h[N];
            uint32_t m[4];
            eight_columns(t[2 * z], t[2 * z + 1], dh);
            keep_masks(a.drop, step, row, j, m);
            if (leaf < 0) m[0] = m[1] = m[2] = m[3] = 0;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float up = bf16_at(v[z], e), d = dh[e] * a.drop.factor;
                float f, df;
                activate_grad(ACT, bf16_at(u[z], e), &f, &df);
                da[e] = d * up * df;
                db[e] = d * f;
                h[e] = f * up * a.drop.factor;
            }
            if (left > 0) {
                put_masked<N>(gate + z * 64, da, m, WHOLE ? N : left);
                put_masked<N>(up_to + z * 64, db, m, WHOLE ? N : left);
                if (a.hidden) put_masked<N>(hidden + z * 64, h, m, WHOLE ? N : left);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

struct Tile {
    int32_t leaf;       // -1: rows of no leaf (their outputs are zero)
    int32_t p0, p1;     // grouped rows: of the tile (forward, dx; int8: plain rows), of the leaf (dw)
    int32_t i0, j0;     // first output row inside the matrix (dw) and first column
    int32_t red, nt;    // summed elements and steps
};

// Tiles go out in eighths: consecutive workgroups sit on the eight XCDs in turn, so XCD x is given
// the x-th eighth (its operands then share that XCD's L2), and its workgroups take it one
// after another; inside it eight row tiles are walked for each column tile.
__device__ __forceinline__ void walk(int64_t t, int64_t nq, int64_t np, int32_t* tq, int32_t* tp) {
    constexpr int G = 8;
    const int64_t band = t / (G * np), r = t - band * G * np;
    const int64_t h = nq - band * G < G ? nq - band * G : G;
    *tp = (int32_t)(r / h);
    *tq = (int32_t)(band * G + r % h);
}

__device__ __forceinline__ Tile uniform(Tile t) {
    int32_t* f = &t.leaf;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Tile) / 4); ++i) f[i] = __builtin_amdgcn_readfirstlane(f[i]);
    return t;
}

constexpr int kScaleBuf = 512;
struct LocateShared {
    int32_t wave_sum[kNT / 64];
    Tile next[2];
};
__device__ __forceinline__ int32_t leaf_start(const ProdArgs& a, int32_t l) {  // inside [0, T] whatever the array holds
    const int64_t o = a.off ? a.off[l] : l ? a.T : 0;
    return (int32_t)(o < 0 ? 0 : o > a.T ? a.T : o);
}
// Rows of entry e: a leaf, or (L, L + 1) the rows after the last and before the first leaf.
__device__ __forceinline__ void entry_rows(const ProdArgs& a, int32_t e, int32_t* b, int32_t* n) {
    *b = e <= a.L ? leaf_start(a, e) : 0;
    *n = (e < a.L ? leaf_start(a, e + 1) : e == a.L ? (int32_t)a.T : leaf_start(a, 0)) - *b;
    if (*n < 0) *n = 0;
}

// Slot of grouped row p, or -1 if the order holds none there.
__device__ __forceinline__ int32_t slot_of(const ProdArgs& a, int32_t p) {
    if (!a.order) return p;
    const int32_t s = a.order[p];
    return s >= 0 && s < a.T ? s : -1;
}

// The query of a slot: slot / fan by a multiplication (slots are below 2^31).
__device__ __forceinline__ uint32_t query_of(const ProdArgs& a, uint32_t s) {
    return (uint32_t)(((uint64_t)s * a.fan_mul) >> a.fan_shift);
}

// Tiles of NQ x NP blocks by a grid of resident workgroups, four waves each, a wave with a
// quarter of the tile (32 NQ x 32 NP); OB bytes an output.  DMA 1: operands are 16-byte aligned with
// whole chunks, and go straight to LDS; otherwise (2 x 2) chunks go through registers, where a
// chunk's missing elements become zero.  DMA 2 (gated): the sum is made of whole steps, two at least, and the row
// side spans less than 4 GB, so that a chunk's address is a uniform one and a 32-bit offset that holds for the whole tile.
//
// Two LDS buffers, one sum step each, and two sets of fragments, 64 bytes of the sum each:
//   first half of step G    multiplies the step's first fragments, reads its second ones
//   barrier                 step G + 1 has landed, nobody reads step G's buffer any more
//   second half             multiplies the second fragments, reads the first ones of step
//                           G + 1, starts the loads of step G + 2 into step G's buffer
// so matrix instructions run through both halves with the LDS reads and the loads issued
// between them.  The steps of a workgroup's tiles form one sequence, so that a tile's
// end costs its stores and nothing else (with more than 254 leaves also its owner's walk over a run of leaf
// starts, find): three cursors walk it, for what is multiplied, what is
// loaded two steps ahead, and the order (rows to gather) three steps ahead.  A tile
// has two steps at least (further ones than its sum has are zeros).
// 4 x 4 (256 x 256, all accumulation registers, one wave a SIMD) loads 64 KB for 512 matrix
// instructions, 3 x 4 an eighth more and 2 x 2 (two workgroups a CU) twice that for each of
// them; tile_shape below chooses.
// Measured: int8 8192 x 4096 x 16384 463-528 us (2.08-2.37 POP/s) of a 484-557 us call; 1000 x 1536 x 100003 to
// float32 256-264 us (400 MB of outputs); bfloat16 32,768 rows of 64 leaves, 1536 -> 4096, 523-589 us (700-790
// TFLOP/s); 16,384 rows of 16 leaves, 1536 x 1536: dx 110-127 us, dw 155-163.  Bound by the power limit and by the
// step's LDS reads: a loop of these matrix instructions alone holds 1.97 GHz on random values (1935 bfloat16
// TFLOP/s; zeros 2.40 GHz), with the LDS reads of a step 1661; the int8 kernel runs at 1.9 GHz, the bfloat16
// one at 1.4 to 1.6.  Without the loads, the barrier or the wait for them (8192 x 6144 x 4096, bfloat16) 360, 422
// and 442 us instead of 446, on zeros 337.
// The gated and 8-bit float products, and what bounds them, stand with their epilogues and half-steps.
template <int MODE, int NQ, int NP, int OB, int DMA>
__global__ __launch_bounds__(kNT, NQ * NP > 4 ? 1 : 2) void prod_tile_kernel(ProdArgs a) {
    constexpr int ELEM = elem_bytes(MODE), FQ = 2 * NQ, FP = 2 * NP, NB = NQ + NP;
    constexpr bool QCOL = MODE == kDw, PCOL = p_by_col(MODE), RAGGED = is_ragged(MODE), PLAIN = is_plain(MODE);
    constexpr bool PERM = kPerm<MODE, OB>, GATE = MODE == kGate, F8 = is_f8(MODE), FAST = DMA == 2;
    constexpr int TQ = NQ * 64, TP = NP * 64 / (GATE ? 2 : 1), STEP = 128 / ELEM;
    constexpr int BUF = NB * kBlock;
    // Steps in LDS at a time: two; float8 at 64 x 64, where a step's matrix instructions (128 clocks a wave) cover nothing of a
    // load's way: four (DMA 3), so that a load has three steps to arrive (1000 x 8192 x 400: 38 us with two, 27 with four; up to
    // eight steps two: 8192 x 128 x 100 4.5 us, with four 6.4).
    constexpr int D = DMA == 3 ? 4 : 2, RING = D * BUF, LOADS = 2 * NB + (F8 ? 1 : 0);
    static_assert(D == 2 || (F8 && NQ * NP == 1));
    static_assert(!F8 || ((TQ > TP ? TQ : TP) * (D - 1) * STEP <= (int)sizeof(zero_rows)));
    // Rows that a thread loads of a row operand's 64, in how many loads: FAST one of 16 bytes of 64, else two of 128.
    constexpr int RH = FAST ? 64 : 32, QS = FAST ? NQ : 2 * NQ;
    constexpr int QR = QCOL ? 2 : PLAIN || FAST ? 1 : 2 * NQ, SLOTS = MODE == kDw ? 2 : QS;
    __shared__ __align__(1024) char lds[(DMA ? D : 1) * BUF];
    __shared__ __align__(16) char turns[OB == 4 && !GATE ? 4 * 16 * kTurnPitch<NP> : 16];
    __shared__ __align__(16) float scales[MODE == kI8 ? 128 * NP + 64 * NQ : F8 ? 64 * NP : 4];
    __shared__ __align__(16) char sbytes[F8 ? D * kScaleBuf : 16];  // float8: a step's scale bytes, Q's 256 and P's
    __shared__ LocateShared sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wq = wave >> 1, wp = wave & 1, g = lane >> 4, li = lane & 15;
    const int32_t np = (int32_t)((a.J + TP - 1) / TP);
    const char* const zero = reinterpret_cast<const char*>(&zero_chunk);

    // Row tiles.  Ragged: a prefix sum of the leaves' row tiles from the leaf starts on the device,
    // one entry or a run of them per thread, kept in registers: this thread's entries have
    // the row tiles [first, last).  Starts in order make at most T / TQ tiles and one more for each entry; starts
    // out of order are held to that, by thread and in all, so that no count passes 32 bits and every
    // tile that is walked belongs to a thread.
    const int32_t E = a.L + 2, run = (E + kNT - 1) / kNT;
    uint32_t first = 0, last = 0;
    int64_t nq = MODE == kDw ? (a.I + TQ - 1) / TQ : (a.T + TQ - 1) / TQ;
    if constexpr (RAGGED) {
        const int32_t whole = (int32_t)(a.T / TQ);
        int32_t sum = 0;
        for (int32_t e = tid * run; e < E && e < (tid + 1) * run; ++e) {
            int32_t b, n;
            entry_rows(a, e, &b, &n);
            sum += (n + TQ - 1) / TQ;
            sum = sum < whole + run ? sum : whole + run;
        }
        last = (uint32_t)wave_inclusive_sum(sum);
        if (lane == 63) sh.wave_sum[wave] = (int32_t)last;
        __syncthreads();
        nq = 0;
#pragma unroll
        for (int w = 0; w < kNT / 64; ++w) {
            const int32_t s = sh.wave_sum[w];
            if (w < wave) last += (uint32_t)s;
            nq += s;
        }
        first = last - (uint32_t)sum;
        nq = nq < whole + E ? nq : whole + E;
        nq = __builtin_amdgcn_readfirstlane((int32_t)nq);
    }
    // dw: a leaf's tiles cost what the leaf has rows, so every XCD takes an eighth of each leaf's tiles (of
    // leaves with fewer than eight, whole leaves).
    const int64_t each = nq * np, eighth = (each + 7) >> 3, total = each * (MODE == kDw ? a.L : 1);
    const bool spread = MODE == kDw && each >= 8;
    const int64_t per = spread ? eighth * a.L : (total + 7) >> 3;
    const int64_t tbeg = (int64_t)(blockIdx.x & 7) * per, tend = spread || tbeg + per < total ? tbeg + per : total;
    auto steps = [&](int32_t red) { return red <= D * STEP ? D : (red + STEP - 1) / STEP; };
    // Publishes tile t in sh.next[k] (to be read after a barrier); past the last one, rows of nothing.
    auto find = [&](int64_t t, int k) {
        int32_t tq, tp;
        if (t >= tend) {
            if (tid == 0) sh.next[k] = Tile{-1, 0, 0, 0, 0, 0, 0x7fffffff};
        } else if constexpr (RAGGED) {
            walk(t, nq, np, &tq, &tp);
            if ((uint32_t)tq >= first && (uint32_t)tq < last) {
                int32_t at = (int32_t)first;
                for (int32_t e = tid * run; e < E && e < (tid + 1) * run; ++e) {
                    int32_t b, n;
                    entry_rows(a, e, &b, &n);
                    const int32_t c = (n + TQ - 1) / TQ;
                    if (tq < at + c) {
                        const int32_t p0 = b + (tq - at) * TQ, p1 = p0 + TQ < b + n ? p0 + TQ : b + n;
                        const int32_t red = e < a.L ? (int32_t)a.red : 0;
                        sh.next[k] = Tile{e < a.L ? e : -1, p0, p1, 0, tp * TP, red, steps(red)};
                        break;
                    }
                    at += c;
                }
            }
        } else if (tid == 0) {
            int32_t leaf = 0;
            int64_t in = t;
            if constexpr (MODE == kDw) {
                leaf = (int32_t)(spread ? (t - tbeg) / eighth : t / each);
                in = spread ? (blockIdx.x & 7) * eighth + (t - tbeg) % eighth : t % each;
            }
            walk(in, nq, np, &tq, &tp);
            if constexpr (MODE == kDw) {
                const int32_t p0 = leaf_start(a, leaf), p1 = leaf_start(a, leaf + 1);
                const int32_t red = p1 > p0 && in < each ? p1 - p0 : 0;
                if (in >= each) tq = (int32_t)nq;  // where eighths do not come out even: past the last row
                sh.next[k] = Tile{leaf, p0, p1, tq * TQ, tp * TP, red, steps(red)};
            } else {
                const int32_t p0 = tq * TQ, p1 = p0 + TQ < a.T ? p0 + TQ : (int32_t)a.T;
                sh.next[k] = Tile{0, p0, p1, 0, tp * TP, (int32_t)a.red, steps((int32_t)a.red)};
            }
        }
    };

    // This thread's 16-byte chunks, two of each block: rows 32 s + rr (of a row operand) or memory rows
    // 32 s + rr (by column), at byte rc or cc of the row.
    auto key = [](int r) { return (r & 3) | (((r >> 2) ^ (r >> 4)) & 1) << 2; };
    auto ckey = [](int r) { return ((r >> 1) & 1) | ((r >> 3) & 1) << 1; };
    const int rr = tid >> 3, rc = ((tid & 7) ^ key(rr)) * 16;
    const int cc = ((((tid & 7) >> 1) ^ ckey(rr)) << 1 | (tid & 1)) * 16;
    // FAST: rows of 64 bytes, chunk c at c ^ turn(row / 4), of PERM column rows (8 a + b) c ^ turn(row / 8).  Of lanes 0-3,
    // 12-15, 20-23 and 24-27 each four rows fill 256 bytes but for the chunk, so turn has to give them four: 0, 3, 2, 1.
    auto turn4 = [](int r) { return -r & 3; };

    Tile w;                               // the tile that is loaded
    const char* qrow[QR];                 // row operand: its rows; by column: this step's memory rows
    const char* prow[MODE == kDw || GATE ? 2 : 1];
    uint32_t poff[PCOL ? (FAST ? NP : 1) : GATE ? (FAST ? NP / 2 : NP) : 2 * NP];  // rows that follow one another: offsets
    uint32_t qoff[PLAIN ? 2 * NQ : FAST ? NQ : 1];  // from prow[0], qrow[0] (FAST: of the blocks, of the rows from a.q)
    int32_t slot[SLOTS];                  // slots of a tile's rows; dw: of the next step's memory rows

    // What the order holds is kept as it was read until it is used, a step later: a check beside the
    // load would wait for it, load by load.
    auto known = [&](int32_t s) { return s >= 0 && s < a.T; };
    // dw: the memory rows of step u of tile n come from the order (load_slots), and are turned into
    // addresses when the step's loads start (set_rows, w being the tile).
    auto load_slots = [&](const Tile& n, int u, int32_t(&to)[SLOTS]) {
        int32_t in[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int32_t r = u * STEP + s * 32 + rr;
            to[s] = in[s] = r < n.red ? n.p0 + r : n.p0 < a.T ? n.p0 : 0;
        }
        if (a.order) {
#pragma unroll
            for (int s = 0; s < 2; ++s) to[s] = a.order[in[s]];
        }
    };
    auto set_rows = [&](int u, const int32_t(&from)[SLOTS]) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const bool is = u * STEP + s * 32 + rr < w.red && known(from[s]);
            qrow[s] = is ? a.q + (int64_t)from[s] * a.qs + (int64_t)w.i0 * 2 + cc : nullptr;
            prow[s] = a.p + (int64_t)query_of(a, (uint32_t)from[s]) * a.ps + (int64_t)w.j0 * 2 + cc;
        }
    };
    // A tile's rows: first what has to be read (slots of its rows, and of lane's and 64 + lane's row of
    // this wave's part, where the results go), later the addresses.
    auto take_rows = [&](const Tile& n, int32_t(&rows)[2]) {
        if constexpr (RAGGED) {
            const int tid = here(threadIdx.x), lane = tid & 63, wq = tid >> 7, rr = tid / (256 / RH);
            const int32_t some = n.p0 < a.T ? n.p0 : 0;  // rows past the tile repeat its first
            int32_t in[QS + 2];
#pragma unroll
            for (int s = 0; s < QS + 2; ++s) {
                const int32_t r = n.p0 + (s < QS ? s * RH + rr : wq * 32 * NQ + (s - QS) * 64 + lane);
                in[s] = r < n.p1 ? r : some;
            }
#pragma unroll
            for (int s = 0; s < QS; ++s) slot[s] = in[s];
#pragma unroll
            for (int u = 0; u < 2; ++u) rows[u] = in[QS + u];
            if (a.order) {
#pragma unroll
                for (int s = 0; s < QS; ++s) slot[s] = a.order[in[s]];
#pragma unroll
                for (int u = 0; u < 2; ++u) rows[u] = a.order[in[QS + u]];
            }
        }
    };
    // Output rows of tile n, of which rows holds what take_rows read; -1: not written.
    auto out_rows = [&](const Tile& n, int32_t(&rows)[2]) {
        const int tid = here(threadIdx.x), lane = tid & 63, wq = tid >> 7;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int32_t i = wq * 32 * NQ + u * 64 + lane;
            if constexpr (MODE == kDw)
                rows[u] = n.i0 + i < a.I ? n.i0 + i : -1;
            else if constexpr (PLAIN)
                rows[u] = n.p0 + i < n.p1 ? n.p0 + i : -1;
            else
                rows[u] = n.p0 + i < n.p1 && known(rows[u]) ? rows[u] : -1;
        }
    };
    auto set_addresses = [&]() {
        const int rr = here(tid) >> 3, r4 = here(tid) >> 2;
        if constexpr (PLAIN) {
            qrow[0] = a.q + w.p0 * a.qs + (F8 ? 0 : rc);
#pragma unroll
            for (int s = 0; s < 2 * NQ; ++s) {
                const int r = s * 32 + rr;
                qoff[s] = (w.p0 + r < w.p1 ? (uint32_t)(r * a.qs) : 0u) + (F8 ? rc : 0);
            }
        } else if constexpr (!QCOL) {
#pragma unroll
            for (int s = 0; s < QS; ++s) {
                int32_t r = known(slot[s]) ? slot[s] : 0;
                if constexpr (MODE == kFwd || GATE) r = (int32_t)query_of(a, (uint32_t)r);
                if constexpr (FAST)  // (a tile without a sum is loaded from zero_rows)
                    qoff[s] = (w.red > 0 ? (uint32_t)((int64_t)r * a.qs) : 0u) + (((tid & 3) ^ turn4(r4 >> 2)) * 16);
                else
                    qrow[s] = a.q + (int64_t)r * a.qs + rc;
            }
        }
        const char* pbase = a.p + (RAGGED && w.leaf > 0 ? w.leaf * a.pg : 0);
        if constexpr (GATE && FAST) {
            // blocks: the gate rows of the tile's columns, then their up rows
            prow[0] = pbase + w.j0 * a.ps;
            prow[1] = prow[0] + a.J * a.ps;
#pragma unroll
            for (int s = 0; s < NP / 2; ++s)
                poff[s] = (w.j0 + s * 64 + r4 < a.J && w.red > 0 ? (uint32_t)((s * 64 + r4) * a.ps) : 0u) +
                          (((tid & 3) ^ turn4(PERM ? r4 >> 3 : r4 >> 2)) * 16);
        } else if constexpr (GATE) {
            // rows of the tile: for each of the wave's columns' halves, 16 NP gate rows, then their up rows
            prow[0] = pbase + w.j0 * a.ps + rc;
            prow[1] = prow[0] + a.J * a.ps;
#pragma unroll
            for (int s = 0; s < NP; ++s) {
                const int r = s * 32 + rr;
                poff[s] = w.j0 + r < a.J ? (uint32_t)(r * a.ps) : 0u;
            }
        } else if constexpr (!PCOL) {
            prow[0] = pbase + w.j0 * a.ps + (F8 ? 0 : rc);
#pragma unroll
            for (int s = 0; s < 2 * NP; ++s) {
                const int r = s * 32 + rr;
                // (a step past the sum of float8 rows comes from zero_rows: rows of one step, or a tile of nothing)
                poff[s] = (w.j0 + r < a.J && (!F8 || w.red > 0) ? (uint32_t)(r * a.ps) : 0u) + (F8 ? rc : 0);
            }
        } else if constexpr (FAST) {
            prow[0] = pbase + (int64_t)w.j0 * 2;
#pragma unroll
            for (int h = 0; h < NP; ++h)  // columns past the last repeat the tile's first; they are not written
                poff[h] = w.red > 0 ? (uint32_t)(rr * a.ps) + (w.j0 + h * 64 + cc / 2 < a.J ? h * 128 + cc : 0) : cc;
        } else if constexpr (MODE != kDw) {
            prow[0] = pbase + rr * a.ps + (int64_t)w.j0 * 2 + cc;
        }
    };
    // Chunk c of a step (of block c / 2, the column side's first): its address, how many bytes of it
    // exist (<= 0: none) and how many of its memory row lie before it.
    auto source = [&](int u, int c, int32_t* valid, int64_t* before) -> const char* {
        const int s = c & 1;
        *before = u * 128 + rc;  // of a row operand
        if (c < 2 * NP) {
            const int h = c >> 1;
            if constexpr (PCOL) *before = (int64_t)w.j0 * 2 + h * 128 + cc;
            if constexpr (GATE) {
                constexpr int H = NP / 2;  // groups of 32 rows of a half
                *valid = w.red * ELEM - (u * 128 + rc);
                return prow[c / H & 1] + poff[c / (2 * H) * H + c % H] + u * 128;
            } else if constexpr (!PCOL) {
                *valid = w.red * ELEM - (u * 128 + rc);
                return prow[0] + poff[c] + u * 128;
            } else if constexpr (MODE != kDw) {
                const int r = u * STEP + s * 32;
                *valid = r + rr < w.red ? ((int32_t)a.J - w.j0) * 2 - (h * 128 + cc) : 0;
                return prow[0] + r * a.ps + h * 128;
            } else {
                *valid = qrow[s] ? ((int32_t)a.J - w.j0) * 2 - (h * 128 + cc) : 0;
                return prow[s] + h * 128;
            }
        } else {
            const int h = (c >> 1) - NP;
            if constexpr (QCOL) *before = (int64_t)w.i0 * 2 + h * 128 + cc;
            if constexpr (!QCOL) {
                *valid = w.red * ELEM - (u * 128 + rc);
                if constexpr (PLAIN)
                    return qrow[0] + qoff[c - 2 * NP] + u * 128;
                else
                    return qrow[c - 2 * NP] + u * 128;
            } else {
                *valid = qrow[s] ? ((int32_t)a.I - w.i0) * 2 - (h * 128 + cc) : 0;
                return qrow[s] + h * 128;
            }
        }
    };

    // Fragments: 16 rows (or columns) x 64 bytes of the sum, in the operand layout of the matrix
    // instruction: lane 16 g + i holds bytes 16 g .. 16 g + 15 of row i.  By column that is eight
    // summed rows, two transposed reads of four.
    const uint32_t base = lds_addr(lds);
    const uint32_t lds_wave = __builtin_amdgcn_readfirstlane(base + wave * 1024);
    // PERM: row 4 a + b of column fragment y is column 32 (y / 2) + 8 a + 4 (y & 1) + b of the part, so
    // that fragments 2 z and 2 z + 1 leave eight consecutive columns in a lane.
    const int pl = PERM ? (li >> 2) * 8 + (li & 3) : li;
    auto row_start = [&](int r, int kk) -> uint32_t { return r * 128 + (((kk * 4 + g) ^ key(r)) * 16); };
    const uint32_t pstart[2] = {base + row_start(wp * 32 * NP + pl, 0), base + row_start(wp * 32 * NP + pl, 1)};
    const uint32_t qstart[2] = {base + NP * kBlock + row_start(wq * 32 * NQ + li, 0),
                                base + NP * kBlock + row_start(wq * 32 * NQ + li, 1)};
    // by column: fragment n of an operand is granule n & 3 of block n >> 2
    const int tr = g * 8 + (li >> 2);
    auto col_start = [&](int n) -> uint32_t {
        return (n >> 2) * kBlock + tr * 128 + (((n & 3) ^ ckey(tr)) * 32) + (li & 3) * 8;
    };
    uint32_t pcol[PCOL ? FP : 1], qcol[QCOL ? FQ : 1];
    if constexpr (PCOL) {
#pragma unroll
        for (int x = 0; x < FP; ++x) pcol[x] = base + col_start(wp * FP + x);
    }
    if constexpr (QCOL) {
#pragma unroll
        for (int x = 0; x < FQ; ++x) qcol[x] = base + NP * kBlock + col_start(wq * FQ + x);
    }
    auto by_row = [&](uint32_t at, uint32_t o) -> v4i { return *(lds_v4i)((lds_char)(uintptr_t)at + o); };
    auto by_col = [&](uint32_t at, uint32_t o) -> v4i {
        const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)((lds_char)(uintptr_t)at + o));
        const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)((lds_char)(uintptr_t)at + o + 512));
        return __builtin_bit_cast(v4i, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto read_p = [&](int x, int kk, uint32_t buf) -> v4i {
        if constexpr (PCOL)
            return by_col(pcol[x] + buf, kk * 4096);
        else if constexpr (PERM)  // four rows on, the key's high bit changes: the other start
            return by_row(pstart[kk ^ (x & 1)] + buf, (x >> 1) * 4096 + (x & 1) * 512);
        else  // 16 rows on likewise
            return by_row(pstart[kk ^ (x & 1)] + buf, x * 2048);
    };
    auto read_q = [&](int x, int kk, uint32_t buf) -> v4i {
        if constexpr (QCOL)
            return by_col(qcol[x] + buf, kk * 4096);
        else
            return by_row(qstart[kk ^ (x & 1)] + buf, x * 2048);
    };

    typedef typename Acc<MODE>::type acc_t;
    acc_t acc[FQ][FP];
    // Two sets of fragments; float8 keeps whole steps: every column fragment, and the row fragments of half-step h.
    v4i pf[F8 ? 1 : 2][F8 ? 1 : FP], qf[F8 ? 1 : 2][F8 ? 1 : FQ];
    v8i p8[F8 ? FP : 1], q8[2][F8 ? FQ / 2 : 1];
    int psc[F8 ? FP : 1], qsc[F8 ? FQ : 1];  // their scale bytes
    const uint32_t sbase = lds_addr(sbytes);
    auto byte_at = [&](uint32_t at) -> int {
        return *(const __attribute__((address_space(3))) uint8_t*)(lds_char)(uintptr_t)at;
    };
    auto read_p8 = [&](int y, int b) {
        p8[y] = halves(read_p(y, 0, b * BUF), read_p(y, 1, b * BUF));
        if constexpr (F8)
            psc[y] = byte_at(sbase + b * kScaleBuf + 256 + wp * 32 * NP + pl + (PERM ? (y >> 1) * 32 + (y & 1) * 4 : y * 16));
    };
    auto read_q8 = [&](int h, int x, int b) {  // x of the half's FQ / 2
        const int n = h * FQ / 2 + x;
        q8[h][x] = halves(read_q(n, 0, b * BUF), read_q(n, 1, b * BUF));
        if constexpr (F8) qsc[n] = byte_at(sbase + b * kScaleBuf + wq * 32 * NQ + n * 16 + li);
    };
    // A step's scale bytes: even waves bring the rows', odd ones the columns' (two waves the same bytes: a branch here would
    // end the matrix instructions' basic block, and the compiler moves them all behind it).  Rows past the last of the
    // pitch repeat its first.
    const int odd = __builtin_amdgcn_readfirstlane(wave & 1);
    const char* const scale_bytes = odd ? a.psc : a.qsc;
    const int64_t scale_pitch = odd ? a.ppitch : a.qpitch;
    auto load_scale_bytes = [&](int u, uint32_t b) {
        if constexpr (F8) {
            const int32_t last = (int32_t)(a.red / STEP) - 1;
            const int64_t r = (odd ? w.j0 : w.p0) + 4 * (int64_t)lane;
            dma4(scale_bytes + (u < last ? u : last) * scale_pitch + (r < scale_pitch ? r : 0),
                 sbase + b * kScaleBuf + odd * 256);
        }
    };
    auto load = [&](int u, int c, uint32_t buf) {
        int32_t valid;
        int64_t before;
        const char* src = source(u, c, &valid, &before);
        dma16(valid > 0 ? src : zero, base + buf + c * 4096 + wave * 1024);
    };
    // FAST.  LDS is a ring of four half-steps (64 bytes of the sum: 4 KB a block).  Half-step h is multiplied from registers
    // while h + 1 is read from the ring and the loads of h + 4 go where h was, so that a load has two to three half-steps to
    // arrive, where two buffers of whole steps give it one to two (16,384 rows, 1536 -> 2 x 4096, without stores: 410 us with two
    // buffers, 380 with the ring, 285 without the loads).  One read or one load stands between two
    // matrix instructions; column fragments are read first, since the next half's first FP instructions use all of them.
    constexpr uint32_t SLOT = NB * 4096;
    const uint32_t qring = base + NP * 4096 + (wq * 32 * NQ + li) * 64 + ((g ^ turn4(li >> 2)) * 16);
    const uint32_t pring = base + (wp * 16 * NP + pl) * 64 + ((g ^ turn4(li >> 2)) * 16);
    uint32_t cring[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) cring[n] = base + (tr * 128 + ((n ^ ckey(tr)) * 32) + (li & 3) * 8);
    auto ring_q = [&](int x, uint32_t at) -> v4i { return by_row(qring + at, x * 1024); };
    auto ring_p = [&](int y, uint32_t at) -> v4i {
        if constexpr (PCOL) {
            const int n = NP == 2 ? y : y & 3;  // fragment wp FP + y: block / 4, granule & 3
            return by_col(cring[n & 3] + at + wp * (FP / 4) * 4096, (y >> 2) * 4096);
        } else {
            const int h = y / NP, f = y % NP;  // gate or up, fragment
            return by_row(pring + at, h * (NP / 2) * 4096 + (PERM ? (f >> 1) * 2048 + (f & 1) * 256 : f * 1024));
        }
    };
    auto ring_load = [&](int u, int half, int c, uint32_t at) {
        if constexpr (FAST) {
            const char* src;
            uint32_t off;
            if (c >= NP) {
                src = a.q + u * 128 + half * 64;
                off = qoff[c - NP];
            } else if constexpr (GATE) {
                src = prow[c / (NP / 2)] + u * 128 + half * 64;
                off = poff[c % (NP / 2)];
            } else {
                src = prow[0] + ((int64_t)u * 64 + half * 32) * a.ps;
                off = poff[c];
            }
            dma16(u * 64 < w.red ? src : reinterpret_cast<const char*>(zero_rows), off, lds_wave + at + c * 4096);
        }
    };
    auto half_ring = [&](int kk, uint32_t from, uint32_t to, int u) {
        constexpr int NM = FQ * FP, NR = FQ + FP;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            acc[m / FP][m % FP] = mma<MODE>(pf[kk][m % FP], qf[kk][m / FP], acc[m / FP][m % FP]);
            const int r = (2 * m * NR + NM - 1) / NM, c = m * NB / NM;  // at most one read (in the first half) and one load
            if (r < NR && r * NM / (2 * NR) == m) {
                if (r >= 1 && r <= FP)
                    pf[kk ^ 1][r - 1] = ring_p(r - 1, from);
                else
                    qf[kk ^ 1][r ? r - FP : 0] = ring_q(r ? r - FP : 0, from);
            }
            if (c < NB && c * NM / NB + NM / (2 * NB) == m) ring_load(u, kk, c, to);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // One half-step: the matrix instructions of fragment set kk; between them the reads of
    // the other set from `buf` and (kk = 1) the loads of step u into the other buffer.
    // float8: half-step kk multiplies half of the row fragments with all column fragments; the first reads the other half,
    // the second, once a column fragment is done with, the next step's, and the first row fragments.  Between two matrix
    // instructions (32 clocks) stands one load or one fragment's reads: in a lump behind every fourth they cost the
    // pipe (8192 x 4096 x 16384, quantising included: 627 us, spread 547).  So that a load is three instructions its address is
    // a uniform one
    // and a lane's offset, the same all along a tile.  That product alone takes 445-515 us (2.1-2.5 PFLOP/s), matrix
    // instructions in 0.54 of the clocks at 1.9-2.0 GHz; without the stores, or without the loads, 60 less.
    auto load8_chunk = [&](int u, int c, uint32_t buf) {
        if constexpr (F8) {
            const bool in = u * STEP < w.red;
            const char* const src = in ? (c < 2 * NP ? prow[0] : qrow[0]) + u * STEP : reinterpret_cast<const char*>(zero_rows);
            dma16(src, c < 2 * NP ? poff[c] : qoff[c - 2 * NP], lds_wave + buf + c * 4096);
        }
    };
    auto half_step8 = [&](int kk, uint32_t buf, int u) {
        constexpr int H = FQ / 2;
        const int b = D == 2 ? (buf ? 1 : 0) : (int)(buf / BUF), bl = D == 2 ? 1 - b : (b + D - 1) % D;  // read, loaded
        const uint32_t to = D == 2 ? BUF - buf : (buf + RING - BUF) % RING;
#pragma unroll
        for (int y = 0; y < FP; ++y) {
#pragma unroll
            for (int x = 0; x < H; ++x) {
                const int n = kk * H + x, at = y * H + x;
                if constexpr (F8) acc[n][y] = mma8<MODE>(p8[y], q8[kk][x], acc[n][y], psc[y], qsc[n]);
                if (kk == 1) {
                    constexpr int S = FP * H;  // evenly: the four waves' 1 KB take the address unit 16 clocks each
#pragma unroll
                    for (int c = 0; c < 2 * NB; ++c)
                        if (c * S / (2 * NB) == at) load8_chunk(u, c, to);
                    if (at == S - 2) load_scale_bytes(u, bl);
                    if (x == H - 1) read_p8(y, b);
                }
                if (x == 0 && y < H) read_q8(kk ^ 1, y, b);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // The second half-step does not use the first's sums: without a use of them here the compiler moves the first's
        // matrix instructions behind the barrier too, whose wait then nothing covers (554 us instead of 513).
        if (kk == 0) {
#pragma unroll
            for (int n = 0; n < H; ++n)
#pragma unroll
                for (int y = 0; y < FP; ++y) {
                    if constexpr (NQ * NP > 4)
                        held(acc[n][y]);
                    else
                        asm volatile("" : "+v"(acc[n][y]));
                }
        }
    };
    auto half_step = [&](int kk, uint32_t buf, int u) {
        constexpr int N = FQ + FP;  // groups: fragments to read, chunks to load
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (n < FQ)
                qf[kk ^ 1][n] = read_q(n, kk ^ 1, buf);
            else
                pf[kk ^ 1][n - FQ] = read_p(n - FQ, kk ^ 1, buf);
            if (kk == 1) load(u, n, BUF - buf);
#pragma unroll
            for (int m = n * FQ * FP / N; m < (n + 1) * FQ * FP / N; ++m)
                acc[m / FP][m % FP] = mma<MODE>(pf[kk][m % FP], qf[kk][m / FP], acc[m / FP][m % FP]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto clear = [&]() {
#pragma unroll
        for (int x = 0; x < FQ * FP; ++x) {
            (&acc[0][0])[x] = acc_t{0, 0, 0, 0};
            if constexpr (NQ * NP > 4) held((&acc[0][0])[x]);
        }
    };
    // int8 scales of tile n: one column and one row of the tile per thread.
    auto load_scales = [&](const Tile& n, float(&v)[3]) {
        const int tid = here(threadIdx.x);
        const int32_t j = n.j0 + tid < a.J ? n.j0 + tid : (int32_t)a.J - 1, r = n.p0 + tid < n.p1 ? n.p0 + tid : n.p0;
        v[1] = a.bias ? a.bias[j] : 0.0f;
        if constexpr (MODE == kI8) {
            v[0] = a.sw[j];
            v[2] = a.sx[r];
        }
    };
    auto keep_scales = [&](const float(&v)[3]) {
        const int tid = here(threadIdx.x);
        if constexpr (F8) {
            if (tid < 64 * NP) scales[tid] = v[1];
            return;
        }
        if (tid < 64 * NP) {
            scales[tid] = v[0];
            scales[64 * NP + tid] = v[1];
        }
        if (tid < 64 * NQ) scales[128 * NP + tid] = v[2];
    };

    // The same straight to LDS (every wave the same): with the values in a register on their way the compiler would wait for
    // it, and so for every load, in each step.  Three steps of at least four follow before they are read.
    auto load_bias = [&](const Tile& n) {
        const int64_t j = n.j0 + lane < a.J ? n.j0 + lane : a.J - 1;
        dma4(a.bias ? reinterpret_cast<const char*>(a.bias + j) : reinterpret_cast<const char*>(zero_rows), lds_addr(scales));
    };

    const uint64_t call_step = is_gated(MODE) && a.drop.t ? step_of_call(a.drop) : 0;
    auto store = [&](const int32_t(&rows)[2], const Tile& n) {
        if constexpr (is_gated(MODE)) {
            auto with = [&](auto act, auto whole) {
                if constexpr (GATE)
                    store_gate<decltype(act)::value, decltype(whole)::value, NQ, NP, OB>(a, acc, rows, n.j0, call_step);
                else
                    store_grad<decltype(act)::value, decltype(whole)::value, NQ, NP>(a, acc, rows, n.leaf, n.j0, call_step);
            };
            auto for_act = [&](auto act) {
                if (n.j0 + TP <= a.J)
                    with(act, std::true_type());
                else
                    with(act, std::false_type());
            };
            if (a.act == AH_SILU)
                for_act(std::integral_constant<int, AH_SILU>());
            else if (a.act == AH_GELU)
                for_act(std::integral_constant<int, AH_GELU>());
            else
                for_act(std::integral_constant<int, AH_RELU>());
        } else
            store_part<MODE, NQ, NP, OB>(a, acc, scales, turns + (OB == 4 ? wave * 16 * kTurnPitch<NP> : 0), rows, n.leaf, n.j0);
    };
    int64_t t = tbeg + (blockIdx.x >> 3);
    const int64_t hop = gridDim.x >> 3;
    if (t >= tend) return;
    find(t, 0);
    __syncthreads();
    if constexpr (DMA) {
        Tile ws = uniform(sh.next[0]);  // the order's cursor: tile, its step, its rows
        int32_t us = 0, rows_s[2] = {};
        int64_t ts = t;
        int k = 1;
        take_rows(ws, rows_s);
        find(ts += hop, k);
        int32_t slot1[SLOTS];
        if constexpr (MODE == kDw) {
            load_slots(ws, 0, slot);
            load_slots(ws, 1, slot1);
        }
        auto advance_order = [&]() {
            if (++us == ws.nt) {
                ws = uniform(sh.next[k]);
                us = 0;
                k ^= 1;
                find(ts += hop, k);
                take_rows(ws, rows_s);
            }
            if constexpr (MODE == kDw) load_slots(ws, us, slot);
        };
        land<0>();
        w = ws;
        int32_t ul = 0, rows_l[2];  // the loads' cursor
#pragma unroll
        for (int u = 0; u < 2; ++u) rows_l[u] = rows_s[u];
        set_addresses();
#pragma unroll
        for (; ul < D; ++ul) {
            if constexpr (MODE == kDw) {
                if (ul == 0)
                    set_rows(0, slot);
                else
                    set_rows(1, slot1);
            }
#pragma unroll
            for (int c = 0; c < 2 * NB; ++c) {
                if constexpr (F8)
                    load8_chunk(ul, c, ul * BUF);
                else if constexpr (FAST)
                    ring_load(ul, c / NB, c % NB, (2 * ul + c / NB) * SLOT);
                else
                    load(ul, c, ul * BUF);
            }
            load_scale_bytes(ul, ul);
        }
        us = D - 1;
        advance_order();
        Tile wc = w;  // what is multiplied
        int32_t uc = 0, rows_c[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) rows_c[u] = rows_l[u];
        clear();
        land<FAST ? 3 * NB : (D - 1) * LOADS>();
        if constexpr (FAST) {
#pragma unroll
            for (int x = 0; x < FQ; ++x) qf[0][x] = ring_q(x, 0);
#pragma unroll
            for (int y = 0; y < FP; ++y) pf[0][y] = ring_p(y, 0);
        } else if constexpr (F8) {
#pragma unroll
            for (int x = 0; x < FQ / 2; ++x) read_q8(0, x, 0);
#pragma unroll
            for (int y = 0; y < FP; ++y) read_p8(y, 0);
        } else {
#pragma unroll
            for (int x = 0; x < FQ; ++x) qf[0][x] = read_q(x, 0, 0);
#pragma unroll
            for (int x = 0; x < FP; ++x) pf[0][x] = read_p(x, 0, 0);
        }
        for (uint32_t cur = 0, next;; cur = next) {
            next = D == 2 ? BUF - cur : (cur + BUF) % RING;
            float sv[3] = {};
            if constexpr (PLAIN) {
                if (uc == 0 && D == 2) load_scales(wc, sv);
            }
            if constexpr (FAST) {
                land<2 * NB>();  // half-step 1 of this step is there; two are in flight
            } else if constexpr (F8) {
                half_step8(0, cur, 0);
                land<(D - 2) * LOADS>();
            } else {
                half_step(0, cur, 0);
                land<0>();
            }
            if constexpr (PLAIN) {
                if (uc == 0) {
                    if constexpr (D > 2)
                        load_bias(wc);
                    else
                        keep_scales(sv);
                }
            }
            if (ul == w.nt) {
                w = ws;
                ul = 0;
#pragma unroll
                for (int u = 0; u < 2; ++u) rows_l[u] = rows_s[u];
                set_addresses();
            }
            if constexpr (MODE == kDw) set_rows(ul, slot);
            advance_order();
            if constexpr (F8) {
                half_step8(1, next, ul++);
            } else if constexpr (FAST) {  // cur: the half-steps of this step, in LDS at cur and cur + SLOT
                half_ring(0, cur + SLOT, cur, ul);
                land<2 * NB>();
                half_ring(1, next, cur + SLOT, ul++);
            } else {
                half_step(1, next, ul++);
            }
            if (++uc < wc.nt) continue;
            if constexpr (NQ * NP > 4 || is_gated(MODE)) settle();
            out_rows(wc, rows_c);
            store(rows_c, wc);
            t += hop;
            if (t >= tend) break;
            wc = w;
            uc = 0;
#pragma unroll
            for (int u = 0; u < 2; ++u) rows_c[u] = rows_l[u];
            clear();
        }
        land<0>();  // no load is left in flight towards LDS
    } else {
        int32_t rows[2] = {};
        v4i stage[2 * NB];
        auto fetch = [&](int u) {
            if constexpr (MODE == kDw) {
                load_slots(w, u, slot);
                set_rows(u, slot);
            }
#pragma unroll
            for (int c = 0; c < 2 * NB; ++c) {
                int32_t valid;
                int64_t before;
                const char* src = source(u, c, &valid, &before);
                stage[c] = load_chunk<ELEM>(src, valid, before);
            }
        };
        for (;;) {
            w = uniform(sh.next[0]);
            if constexpr (MODE == kI8) {
                float sv[3];
                load_scales(w, sv);
                keep_scales(sv);
            }
            take_rows(w, rows);
            set_addresses();
            clear();
            fetch(0);
            for (int u = 0; u < w.nt; ++u) {
                __syncthreads();
#pragma unroll
                for (int c = 0; c < 2 * NB; ++c) *reinterpret_cast<v4i*>(lds + c * 4096 + tid * 16) = stage[c];
                __syncthreads();
                if (u + 1 < w.nt) fetch(u + 1);
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                    for (int x = 0; x < FQ; ++x) qf[kk][x] = read_q(x, kk, 0);
#pragma unroll
                    for (int x = 0; x < FP; ++x) pf[kk][x] = read_p(x, kk, 0);
#pragma unroll
                    for (int m = 0; m < FQ * FP; ++m)
                        acc[m / FP][m % FP] = mma<MODE>(pf[kk][m % FP], qf[kk][m / FP], acc[m / FP][m % FP]);
                }
            }
            out_rows(w, rows);
            if constexpr (is_gated(MODE)) settle();
            store(rows, w);
            t += hop;
            if (t >= tend) break;
            __syncthreads();
            find(t, 0);
            __syncthreads();
        }
    }
}

// Tokens to int8 codes: step = max |x| / 127 (float32), code = rint(x / step), the division IEEE.
// A row with a NaN or an infinity gets step NaN and zero codes, so that it spoils its own
// outputs and no others.
template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    if constexpr (sizeof(T) == 4)
        return __builtin_bit_cast(float, v);
    else
        return __uint_as_float((uint32_t)v << 16);
}
// Largest |x| of a chunk, +inf where one is NaN or infinite.
template <typename T>
__device__ __forceinline__ float chunk_max(v4i v) {
    constexpr int NV = 16 / sizeof(T);
    T e[NV];
    __builtin_memcpy(e, &v, 16);
    float m = 0.0f;
    bool bad = false;
#pragma unroll
    for (int r = 0; r < NV; ++r) {
        const float f = fabsf(to_f32(e[r]));
        bad |= !(f < INFINITY);
        m = fmaxf(m, f);
    }
    return bad ? INFINITY : m;
}
// rint(x / s) for the elements of a chunk.  With inv = 1 / s, t = x inv is off from the quotient by less than
// 2.3e-5 (|x / s| <= 127, three roundings of 2^-24), so where t lies further than 5e-5 from the middle between
// whole numbers rint(t) is rint of the IEEE quotient; else, or where 1 / s overflows, the chunk is
// divided (one in 600 chunks of 8).
template <typename T>
__device__ __forceinline__ void chunk_codes(v4i v, float s, float inv, int8_t* q) {
    constexpr int NV = 16 / sizeof(T);
    T e[NV];
    __builtin_memcpy(e, &v, 16);
    float n[NV], off = 0.0f;
#pragma unroll
    for (int r = 0; r < NV; ++r) {
        const float t = to_f32(e[r]) * inv;
        n[r] = rintf(t);
        off = fmaxf(off, fabsf(t - n[r]));
    }
    if (!(off < 0.49995f) || !(s > 1e-37f)) {
#pragma unroll
        for (int r = 0; r < NV; ++r) n[r] = s > 0.0f ? rintf(to_f32(e[r]) / s) : 0.0f;
    }
#pragma unroll
    for (int r = 0; r < NV; ++r) q[r] = (int8_t)(int)fminf(fmaxf(n[r], -127.0f), 127.0f);
}
__device__ __forceinline__ float step_of(float m) { return m < INFINITY ? m / 127.0f : NAN; }

// Few rows: the product is a single pass over the weights.  A workgroup has 16 columns of one matrix and 16 FR
// rows at a time; its eight waves share out the sum, load their pieces of both operands from
// memory into the matrix instruction's layout (lane 16 g + i: 16 bytes of row i), 4 x 64 bytes at once,
// and add up through LDS in a fixed order.  XB = 2 or 4: Q holds tokens of that many bytes an
// element, which every workgroup quantises for itself (as i8_quantize_kernel does, bit for bit).
// HBM-bound in the weights where they are many: 64 slots of 64 leaves, 1536 x 1536, 189 MB of weights
// in 34 us for grouping and product (5.6 TB/s); one token, 1536 -> 4096, 9.5 us a call, a launch's
// latency (7.0 on the GPU; 15.6 with tiles and quantising in a launch of its own).
constexpr int kRowWaves = 8;
// STRIP (gated sums of at most 512 bytes, eight pieces): nothing to share out, so every wave has 16 columns of its own and the
// whole sum (999 slots of 37 leaves, 100 -> 2 x 385, on the GPU: 12.1 us, 18 with the sum shared by eight waves).  Bound
// by the chain of leaf starts, order, row and weights, each a load that waits for the one before, and by the epilogue
// (with silu in gelu's place 9.8; a Philox call makes eight numbers of which a lane uses four).  One token, 1536 ->
// 2 x 4096, shares the sum: 7.5 us, of which 25 MB of weights are 4.7.
template <int MODE, int FR, bool WHOLE, int XB, bool STRIP = false>
__global__ __launch_bounds__(kRowWaves * 64) void prod_rows_kernel(ProdArgs a) {
    constexpr int ELEM = elem_bytes(MODE), U = STRIP ? 2 : 4, G = MODE == kGate ? 2 : 1;
    static_assert(XB == 0 || (MODE == kI8 && FR == 1 && WHOLE), "");
    typedef typename Acc<MODE>::type acc_t;
    __shared__ acc_t part[STRIP ? 1 : kRowWaves][STRIP ? 1 : G * FR][64];
    __shared__ float most[kRowWaves][16];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, li = lane & 15;
    const int32_t kb = (int32_t)a.red * ELEM, steps = (kb + 63) >> 6;
    const int32_t s0 = STRIP ? 0 : steps * wave / kRowWaves, s1 = STRIP ? steps : steps * (wave + 1) / kRowWaves;
    const int32_t strip = STRIP ? blockIdx.x * kRowWaves + wave : blockIdx.x;
    const int32_t j = strip * 16 + g * 4;  // this lane's four output columns
    const int32_t leaf = MODE == kI8 ? 0 : blockIdx.y;
    const uint64_t call_step = MODE == kGate && a.drop.t ? step_of_call(a.drop) : 0;
    auto put = [&](int32_t row, v4f v) {
        if (a.out_f32) {
            float* o = static_cast<float*>(a.out) + row * a.J + j;
            if (j + 4 <= a.J)
                __builtin_memcpy(o, &v, 16);
            else if (j < a.J)
                store_left<4>(reinterpret_cast<char*>(o), __builtin_bit_cast(v4i, v), (int32_t)a.J - j);
        } else {
            uint16_t* o = static_cast<uint16_t*>(a.out) + row * a.J + j;
            const uint32_t w[2] = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
            if (j + 4 <= a.J)
                __builtin_memcpy(o, w, 8);
            else if (j < a.J)
                store_left<2>(reinterpret_cast<char*>(o), v4i{(int)w[0], (int)w[1], 0, 0}, (int32_t)a.J - j);
        }
    };
    int32_t p0, p1;
    if constexpr (MODE == kI8) {
        p0 = blockIdx.y * 16 * FR;
        p1 = p0 + 16 * FR < a.T ? p0 + 16 * FR : (int32_t)a.T;
    } else if (leaf < a.L) {
        p0 = leaf_start(a, leaf);
        p1 = leaf_start(a, leaf + 1);
    } else {  // rows of no leaf
        if (blockIdx.z > 0) return;
        const int32_t head = leaf_start(a, 0), tail = leaf_start(a, a.L);
        for (int32_t p = (STRIP ? lane : tid) >> 2; p < head + (int32_t)a.T - tail; p += (STRIP ? 1 : kRowWaves) * 16) {
            const int32_t row = slot_of(a, p < head ? p : tail + p - head), c = strip * 16 + (tid & 3) * 4;
            if (row < 0 || c >= a.J) continue;
            const int32_t left = (int32_t)a.J - c, ob = a.out_f32 ? 4 : 2;
            char* o = static_cast<char*>(a.out) + (row * a.J + c) * ob;
            for (int32_t e = 0; e < (left < 4 ? left : 4) * ob; e += 2) *reinterpret_cast<uint16_t*>(o + e) = 0;
            if (MODE == kGate && a.pre) {
                const float none[4] = {};
                char* const p = a.pre + ((int64_t)row * 2 * a.J + c) * 2;
                put_bf16(p, none, left);
                put_bf16(p + a.J * 2, none, left);
            }
        }
        return;
    }
    if (STRIP && strip * 16 >= a.J) return;
    const int32_t col = strip * 16 + li < a.J ? strip * 16 + li : (int32_t)a.J - 1;
    const char* const prow = a.p + leaf * a.pg + col * a.ps;
    auto fetch = [&](const char* row, int32_t o) -> v4i {
        v4i v = {0, 0, 0, 0};
        if constexpr (WHOLE) {
            if (o < kb) v = *reinterpret_cast<const v4i*>(row + o);
        } else if (o < kb) {  // the last chunk is read as the row's last 16 bytes
            const int cut = o + 16 > kb ? o + 16 - kb : 0;
            __builtin_memcpy(&v, row + o - cut, 16);
            v = shift_down(v, cut);
        }
        return v;
    };
    // the output's scales, asked for before the operands: at the end they would cost another trip
    float sw[4] = {}, bias[4] = {};
    if constexpr (MODE == kI8) {
        if (wave < FR) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int32_t je = j + e < a.J ? j + e : (int32_t)a.J - 1;
                sw[e] = a.sw[je];
                bias[e] = a.bias ? a.bias[je] : 0.0f;
            }
        }
    }
    for (int32_t p = p0 + blockIdx.z * 16 * FR; p < p1; p += gridDim.z * 16 * FR) {
        int32_t out_row[FR];
        const char* qrow[FR];
        float sx = 0.0f;  // of the rows that this wave stores (fragment `wave`)
#pragma unroll
        for (int f = 0; f < FR; ++f) {
            int32_t r = p + f * 16 + li;
            const bool in = r < p1;
            if (!in) r = p;  // rows past the last repeat the first; they are not written
            if constexpr (MODE == kI8) {
                out_row[f] = in ? r : -1;
                if (XB == 0 && wave == f) sx = a.sx[r];
            } else {
                r = slot_of(a, r);
                out_row[f] = in ? r : -1;
                r = r < 0 ? 0 : (int32_t)query_of(a, (uint32_t)r);
            }
            qrow[f] = a.q + (int64_t)r * a.qs;
        }
        v4i pv[U], uv[G == 2 ? U : 1], qv[U][FR], xv[XB > 0 ? U : 1][XB > 0 ? XB : 1];
        auto load = [&](int32_t s) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s + u < s1) {
                    const int32_t o = (s + u) * 64 + g * 16;
                    if constexpr (XB == 0) {
#pragma unroll
                        for (int f = 0; f < FR; ++f) qv[u][f] = fetch(qrow[f], o);
                    } else {
#pragma unroll
                        for (int c = 0; c < XB; ++c)
                            xv[u][c] = o < kb ? *reinterpret_cast<const v4i*>(qrow[0] + (o * XB + c * 16)) : v4i{0, 0, 0, 0};
                    }
                    pv[u] = fetch(prow, o);
                    if constexpr (G == 2) uv[u] = fetch(prow + a.J * a.ps, o);
                }
        };
        load(s0);
        if constexpr (XB > 0) {
            float m = 0.0f;
            auto look = [&](v4i v) {
                if constexpr (XB == 2)
                    m = fmaxf(m, chunk_max<uint16_t>(v));
                else
                    m = fmaxf(m, chunk_max<float>(v));
            };
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s0 + u < s1) {
#pragma unroll
                    for (int c = 0; c < XB; ++c) look(xv[u][c]);
                }
            for (int32_t s = s0 + U; s < s1; ++s) {
                const int32_t o = s * 64 + g * 16;
                if (o < kb) {
#pragma unroll
                    for (int c = 0; c < XB; ++c) look(*reinterpret_cast<const v4i*>(qrow[0] + (o * XB + c * 16)));
                }
            }
            m = fmaxf(m, __shfl_xor(m, 16, 64));
            m = fmaxf(m, __shfl_xor(m, 32, 64));
            most[wave][li] = m;
            __syncthreads();
            m = most[0][li];
#pragma unroll
            for (int w = 1; w < kRowWaves; ++w) m = fmaxf(m, most[w][li]);
            sx = step_of(m);
        }
        acc_t acc[G * FR];
#pragma unroll
        for (int f = 0; f < G * FR; ++f) acc[f] = acc_t{0, 0, 0, 0};
        for (int32_t s = s0; s < s1; s += U) {
            if (s > s0) load(s);
            if constexpr (XB > 0) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (s + u < s1) {
                        int8_t q[16];
#pragma unroll
                        for (int c = 0; c < XB; ++c) {
                            if constexpr (XB == 2)
                                chunk_codes<uint16_t>(xv[u][c], sx, 1.0f / sx, q + c * 8);
                            else
                                chunk_codes<float>(xv[u][c], sx, 1.0f / sx, q + c * 4);
                        }
                        __builtin_memcpy(&qv[u][0], q, 16);
                    }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s + u < s1) {
#pragma unroll
                    for (int f = 0; f < FR; ++f) {
                        acc[f] = mma<MODE>(pv[u], qv[u][f], acc[f]);
                        if constexpr (G == 2) acc[FR + f] = mma<MODE>(uv[u], qv[u][f], acc[FR + f]);
                    }
                }
        }
        if constexpr (!STRIP) {
#pragma unroll
            for (int f = 0; f < G * FR; ++f) part[wave][f][lane] = acc[f];
            __syncthreads();
        }
        auto sum_of = [&](int f) {
            if constexpr (STRIP) return acc[f];
            acc_t t = part[0][STRIP ? 0 : f][lane];
#pragma unroll
            for (int w = 1; w < kRowWaves; ++w) t += part[STRIP ? 0 : w][STRIP ? 0 : f][lane];
            return t;
        };
#pragma unroll
        for (int f = 0; f < FR; ++f)
            if ((STRIP || wave == f) && out_row[f] >= 0) {
                const acc_t t = sum_of(f);
                v4f v;
                if constexpr (MODE == kI8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = (float)t[e] * sx * sw[e];
                        if (a.bias) v[e] += bias[e];
                    }
                } else if constexpr (G == 2) {
                    const v4f up = sum_of(FR + f);
                    float drop[4];
                    dropout_factors(a.drop, call_step, out_row[f], j, drop);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = dropped(activate(a.act, t[e]) * up[e], drop[e]);
                    if (a.pre) {
                        const float gates[4] = {t[0], t[1], t[2], t[3]}, ups[4] = {up[0], up[1], up[2], up[3]};
                        char* const p = a.pre + ((int64_t)out_row[f] * 2 * a.J + j) * 2;
                        put_bf16(p, gates, (int32_t)a.J - j);
                        put_bf16(p + a.J * 2, ups, (int32_t)a.J - j);
                    }
                } else {
                    v = t;
                }
                put(out_row[f], v);
            }
        if (!STRIP && p + (int32_t)gridDim.z * 16 * FR < p1) __syncthreads();
    }
}

inline bool chunked(const void* p, int64_t stride_bytes, int64_t width_bytes) {
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride_bytes | (uintptr_t)width_bytes) & 15) == 0;
}

// Row tiles of TQ rows (ragged: their number is known on the device only; `most` bounds it, the
// estimate takes every leaf to end inside a tile).
template <int MODE>
int64_t row_tiles(const ProdArgs& a, int64_t TQ, bool most) {
    if (MODE == kDw) return (a.I + TQ - 1) / TQ * a.L;
    if (is_plain(MODE)) return (a.T + TQ - 1) / TQ;
    return a.T / TQ + (most ? a.L + 2 : (a.T < a.L ? a.T : a.L) / 2 + 1);
}

// Blocks of the tile's row side: 4 (of 4 x 4), 3 (of 3 x 4) or 2 (of 2 x 2).  The time is taken as the
// rounds that the resident workgroups go through times a round's blocks a CU, over the shape's
// rate on large products (1, 0.97 and 0.85: 32,768 rows of 64 leaves, 1536 -> 4096: 560, 582 and
// 650 us, where rounds and ragged ends explain the first ratio).  dw always takes 2 x 2: its tiles are as
// unequal as the leaves (16 leaves of 450 to 1,900 rows, 1536 x 1536, with dx: 302 us; 3 x 4 by a
// workgroup for each tile 314, by resident workgroups 334).
template <int MODE>
int tile_shape(const ProdArgs& a) {
    auto time = [&](int64_t TQ, int64_t TP, int64_t resident, double round) {
        return (double)((row_tiles<MODE>(a, TQ, false) * ((a.J + TP - 1) / TP) + resident - 1) / resident) * round;
    };
    const double t4 = time(256, 256, kCUs, 16), t3 = time(192, 256, kCUs, 12 / 0.97),
                 t2 = time(128, 128, 2 * kCUs, 8 / 0.85);
    return t2 <= t3 && t2 <= t4 ? 2 : t3 < t4 ? 3 : 4;
}

// The same for gated and 8-bit float products, whose tiles end in epilogues of their own weight and whose sums may be long
// over few tiles: a round of the resident workgroups takes (steps of its sum) x step + end, and, with two workgroups a CU, a
// last round of one a CU the share `alone` of that.  Measured, us:
//   8-bit float           4 x 4   3 x 4   4 x 3   2 x 3   2 x 2   1 x 1
//   8192 x 4096 x 16384     461     501     509     637     544    1248
//   8192 x 4096 x 1536       52      82      46      59      57     119
//   1536 x 8192 x 4096       90      74      74     105      60     113
//   4096 x 8192 x 1536       92      76      75      57      60     115
//   16384 x 1024 x 2048      48      49      49      57      44      91
//   2048 x 4096 x 1536       50      41      41      31      27      39
//   333 x 4096 x 1001        52      42      43      29      23      17
//   gate, rows of 16 leaves                4 x 4   3 x 4   2 x 2      gradient   3 x 4   2 x 2
//   16384, 1536 -> 2 x 4096                  553     609     645                   386     439
//   16384, 768 -> 2 x 1024                   107      91      79                    79      69
//   4096, 1536 -> 2 x 2048                   115     101      84                    59      68
// The figures below are fits to these and to more sizes.
struct TileCost {
    int nq, np, per_cu;
    double step, end, alone;  // us, us, share
};
template <int MODE, int N>
int cheapest(const ProdArgs& a, const TileCost (&shapes)[N], int64_t J, int64_t steps, double* least_time = nullptr) {
    int best = 0;
    double least = 0.0;
    for (const auto& s : shapes) {
        const int64_t TQ = s.nq * 64, TP = s.np * 64;
        // every second leaf ends inside a tile of its own
        const int64_t ends = is_plain(MODE) ? 0 : (a.T < a.L ? a.T : a.L) / 2;
        const int64_t tiles = ((a.T + TQ - 1) / TQ + ends) * ((J + TP - 1) / TP);
        const int64_t resident = (int64_t)kCUs * s.per_cu, rest = tiles % resident;
        const double rounds = (double)(tiles / resident) + (rest == 0 ? 0.0 : rest <= kCUs ? s.alone : 1.0);
        const double time = rounds * ((double)steps * s.step + s.end);
        if (best == 0 || time < least) {
            best = s.nq * 10 + s.np;
            least = time;
        }
    }
    if (least_time) *least_time = least;
    return best;
}
template <int MODE>
int f8_shape(const ProdArgs& a, double* time = nullptr) {
    const TileCost shapes[] = {{4, 4, 1, 1.45, 11.0, 1.0}, {3, 4, 1, 1.21, 6.7, 1.0}, {4, 3, 1, 1.21, 6.7, 1.0},
                               {2, 3, 1, 0.84, 3.0, 1.0},  {2, 2, 2, 0.96, 3.3, 0.7},  {1, 1, 2, 0.57, 3.0, 0.65}};
    return cheapest<MODE>(a, shapes, a.J, (a.red + 127) / 128, time);
}
template <int MODE>
int gated_shape(const ProdArgs& a) {
    const int64_t steps = (a.red + 63) / 64;
    if constexpr (MODE == kGate) {
        const TileCost f32[] = {{3, 4, 1, 1.65, 10.5, 1.0}, {2, 2, 2, 1.32, 4.0, 0.5}};  // (4 x 4 would spill registers)
        if (a.out_f32) return cheapest<MODE>(a, f32, 2 * a.J, steps);
        const TileCost shapes[] = {f32[0], f32[1], {4, 4, 1, 2.1, 10.0, 1.0}};
        return cheapest<MODE>(a, shapes, 2 * a.J, steps);
    } else {
        const TileCost shapes[] = {{3, 4, 1, 2.0, 14.5, 1.0}, {2, 2, 2, 1.55, 12.5, 0.45}};
        return cheapest<MODE>(a, shapes, a.J, steps);
    }
}

template <int MODE, int NQ, int NP, int DMA>
hipError_t launch_tiles(const ProdArgs& a, hipStream_t stream) {
    constexpr int TQ = NQ * 64, TP = NP * 64 / (MODE == kGate ? 2 : 1);
    const int64_t np = (a.J + TP - 1) / TP, each = row_tiles<MODE>(a, TQ, true) * np;
    const int64_t resident = kCUs * (NQ * NP > 4 ? 1 : 2);
    int64_t wgs = (each + 7) / 8 * 8;
    if (MODE == kDw) {  // a workgroup for each tile: they are of unequal length, and start as others end
        const int64_t leaf = (a.I + TQ - 1) / TQ * np;
        if (leaf >= 8) wgs = (leaf + 7) / 8 * 8 * a.L;
    }
    if ((MODE != kDw || wgs * kNT > kMaxGridItems) && wgs > resident) wgs = resident;
    const dim3 grid((uint32_t)wgs);
    if constexpr (MODE != kGrad && !(MODE == kGate && NQ == 4)) {
        if (a.out_f32) {
            hipLaunchKernelGGL((prod_tile_kernel<MODE, NQ, NP, 4, DMA>), grid, dim3(kNT), 0, stream, a);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((prod_tile_kernel<MODE, NQ, NP, 2, DMA>), grid, dim3(kNT), 0, stream, a);
    return hipGetLastError();
}

// Whether prod_rows_kernel's grid, a workgroup for every 16 columns, can be launched; the tiled kernel takes
// any number of columns.
inline bool rows_launchable(int64_t J) { return (J + 15) / 16 * (kRowWaves * 64) <= kMaxGridItems; }

// Row fragments of prod_rows_kernel, or 0 for the tiled kernel.
template <int MODE>
int row_fragments(const ProdArgs& a) {
    const int64_t rows = MODE == kI8 ? a.T : (a.T + a.L - 1) / a.L;  // of one matrix, on average
    if (!rows_launchable(a.J)) return 0;
    if (a.L >= 65535 || a.red * (MODE == kI8 ? 1 : 2) < 16) return 0;  // the grid's second dimension; a row's last 16 bytes
    if (MODE == kI8) return rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= 64 ? 4 : 0;
    return rows <= 6 ? 1 : rows <= 14 ? 2 : rows <= 48 ? 4 : 0;  // leaves differ: room for twice the average
}

template <int MODE, int FR, int XB = 0>
hipError_t launch_rows(const ProdArgs& a, bool whole, hipStream_t stream) {
    // a leaf's rows beyond 16 FR go to a second workgroup
    const dim3 grid((uint32_t)((a.J + 15) / 16), (uint32_t)(MODE == kI8 ? (a.T + 16 * FR - 1) / (16 * FR) : a.L + 1),
                    MODE == kI8 || a.T / a.L < 8 ? 1 : 2);
    if constexpr (MODE == kGate) {
        if (a.red * 2 <= kRowWaves * 64) {
            const dim3 strips((grid.x + kRowWaves - 1) / kRowWaves, grid.y, grid.z);
            auto kernel = whole ? prod_rows_kernel<MODE, FR, true, 0, true> : prod_rows_kernel<MODE, FR, false, 0, true>;
            hipLaunchKernelGGL(kernel, strips, dim3(kRowWaves * 64), 0, stream, a);
            return hipGetLastError();
        }
    }
    if constexpr (XB == 0) {
        if (!whole) {
            hipLaunchKernelGGL((prod_rows_kernel<MODE, FR, false, 0>), grid, dim3(kRowWaves * 64), 0, stream, a);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((prod_rows_kernel<MODE, FR, true, XB>), grid, dim3(kRowWaves * 64), 0, stream, a);
    return hipGetLastError();
}

// Gated products without FAST loads: 2 x 2 tiles, or, where those leave half the chip without one, 1 x 1 (gate: 1 x 2, of 64
// columns), whose workgroups go through a quarter (half) of the epilogue each (1,500 rows of 21 leaves, 77 -> 200: gradient 16.0 us
// -> 8.9, 77 -> 2 x 200 10.8 -> 8.5; 1,000 rows, 768 -> 2048: gradient 23 -> 17).
template <int MODE, int DMA>
hipError_t launch_small(const ProdArgs& a, hipStream_t stream) {
    const int64_t J = MODE == kGate ? 2 * a.J : a.J;
    if (row_tiles<MODE>(a, 128, false) * ((J + 127) / 128) <= kCUs)
        return launch_tiles<MODE, 1, MODE == kGate ? 2 : 1, DMA>(a, stream);
    return launch_tiles<MODE, 2, 2, DMA>(a, stream);
}

template <int MODE>
hipError_t launch_prod(ProdArgs a, int32_t fan, hipStream_t stream) {
    const int e = elem_bytes(MODE);
    bool whole;
    if (MODE == kDw)
        whole = chunked(a.q, a.qs, a.I * e) && chunked(a.p, a.ps, a.J * e);
    else if (MODE == kDx || MODE == kGrad)
        whole = chunked(a.q, a.qs, a.red * e) && chunked(a.p, a.ps, a.J * e);
    else
        whole = chunked(a.q, a.qs, a.red * e) && chunked(a.p, a.ps, 0);
    // ceil(2^(31 + l) / fan) with l = ceil(log2 fan) divides every slot below 2^31 exactly
    int l = 0;
    while (((int64_t)1 << l) < fan) ++l;
    a.fan_shift = 31 + l;
    a.fan_mul = (uint32_t)((((uint64_t)1 << (31 + l)) + fan - 1) / fan);
    const int64_t pitch = a.J * (a.out_f32 ? 4 : 2);
    a.bypass = MODE != kFwd && !is_gated(MODE) && ((reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)pitch) & 63) == 0;
    if constexpr (MODE == kI8 || MODE == kFwd || MODE == kGate) {
        switch (row_fragments<MODE>(a)) {
            case 1: return launch_rows<MODE, 1>(a, whole, stream);
            case 2: return launch_rows<MODE, 2>(a, whole, stream);
            case 4: return launch_rows<MODE, 4>(a, whole, stream);
        }
    }
    if constexpr (is_gated(MODE)) {
        if (!whole) return launch_small<MODE, 0>(a, stream);
    } else if constexpr (!is_f8(MODE)) {
        if (!whole) return launch_tiles<MODE, 2, 2, 0>(a, stream);
    }
    if constexpr (MODE == kDw) {
        return launch_tiles<MODE, 2, 2, 1>(a, stream);
    } else if constexpr (is_gated(MODE)) {
        // Other sums (and more than 4 GB of rows) take the general loads, at the smallest tile.
        if (a.red % 64 != 0 || a.red < 128 || a.T / fan * a.qs >= ((int64_t)1 << 32))
            return launch_small<MODE, 1>(a, stream);
        switch (gated_shape<MODE>(a)) {
            case 44:
                if constexpr (MODE == kGate) return launch_tiles<MODE, 4, 4, 2>(a, stream);
            case 34: return launch_tiles<MODE, 3, 4, 2>(a, stream);
            default: return launch_small<MODE, 1>(a, stream);  // (with the ring's barriers 12 % slower)
        }
    } else if constexpr (is_f8(MODE)) {
        switch (f8_shape<MODE>(a)) {
            case 44: return launch_tiles<MODE, 4, 4, 1>(a, stream);
            case 34: return launch_tiles<MODE, 3, 4, 1>(a, stream);
            case 43: return launch_tiles<MODE, 4, 3, 1>(a, stream);
            case 23: return launch_tiles<MODE, 2, 3, 1>(a, stream);
            case 11: return a.red > 8 * 128 ? launch_tiles<MODE, 1, 1, 3>(a, stream) : launch_tiles<MODE, 1, 1, 1>(a, stream);
            default: return launch_tiles<MODE, 2, 2, 1>(a, stream);
        }
    } else {
        switch (tile_shape<MODE>(a)) {
            case 4: return launch_tiles<MODE, 4, 4, 1>(a, stream);
            case 3: return launch_tiles<MODE, 3, 4, 1>(a, stream);
            default: return launch_tiles<MODE, 2, 2, 1>(a, stream);
        }
    }
}

}  // namespace
}  // namespace ah
