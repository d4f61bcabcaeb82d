// Matrix products of a learned query side on the CDNA4 matrix cores: int8 rows
// with a scale for each token and channel, and bfloat16 rows grouped by leaf
// (every leaf of a partition has its own weight matrix) with their gradients.
//
// All of them are one contraction, out[i][j] = sum_t Q[i][t] P[j][t], with Q the
// row side (tokens) and P the column side (channels):
//   int8     Q = codes [m][k],           P = codes [n][k]            t = k
//   forward  Q = queries of a leaf,      P = the leaf's W [n][k]     t = k
//   dx       Q = slot gradients,         P = the leaf's W, by column t = n
//   dw       Q = slot gradients by column, P = queries by column     t = the leaf's rows
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
#include "ah_device.hpp"
#include "ah_kernels.hpp"
#include "../../include/ah.h"

namespace ah {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

enum { kI8 = 0, kFwd = 1, kDx = 2, kDw = 3 };

constexpr int kNT = 256;     // threads: 2 x 2 waves
constexpr int kCUs = 256;    // compute units of an MI355X (a multiple of its 8 XCDs)
constexpr int kBlock = 8192; // bytes of a block

// Source of chunks that lie outside an operand (past its sum or its columns).
__device__ const v4i zero_chunk = {0, 0, 0, 0};

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
    int32_t bypass;        // rows of whole 64-byte sectors
    const float *sx, *sw, *bias;  // int8
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
constexpr bool kPerm = OB == 2 && MODE < kDx;
template <int NP>
constexpr int kTurnCols = NP == 2 ? 32 : 64;
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
                for (int e = 0; e < N / 2; ++e) w[e] = bf16_bits(v[2 * e]) | bf16_bits(v[2 * e + 1]) << 16;
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

struct LocateShared {
    int32_t wave_sum[kNT / 64];
    Tile next[2];
};
__device__ __forceinline__ int32_t leaf_start(const ProdArgs& a, int32_t l) {  // inside [0, T] whatever the array holds
    const int64_t o = a.off[l];
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
// quarter of the tile (32 NQ x 32 NP); OB bytes an output.  DMA: operands are 16-byte aligned with
// whole chunks, and go straight to LDS; otherwise (2 x 2) chunks go through registers, where a
// chunk's missing elements become zero.
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
template <int MODE, int NQ, int NP, int OB, bool DMA>
__global__ __launch_bounds__(kNT, NQ * NP > 4 ? 1 : 2) void prod_tile_kernel(ProdArgs a) {
    constexpr int ELEM = MODE == kI8 ? 1 : 2, FQ = 2 * NQ, FP = 2 * NP, NB = NQ + NP;
    constexpr bool QCOL = MODE == kDw, PCOL = MODE >= kDx, RAGGED = MODE == kFwd || MODE == kDx;
    constexpr bool PERM = kPerm<MODE, OB>;
    constexpr int TQ = NQ * 64, TP = NP * 64, STEP = 128 / ELEM;
    constexpr int BUF = NB * kBlock;
    constexpr int QR = QCOL ? 2 : MODE == kI8 ? 1 : 2 * NQ, SLOTS = MODE == kDw ? 2 : 2 * NQ;
    __shared__ __align__(1024) char lds[(DMA ? 2 : 1) * BUF];
    __shared__ __align__(16) char turns[OB == 4 ? 4 * 16 * kTurnPitch<NP> : 16];
    __shared__ __align__(16) float scales[MODE == kI8 ? 128 * NP + 64 * NQ : 4];
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
    auto steps = [&](int32_t red) { return red <= 2 * STEP ? 2 : (red + STEP - 1) / STEP; };
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

    Tile w;                               // the tile that is loaded
    const char* qrow[QR];                 // row operand: its rows; by column: this step's memory rows
    const char* prow[MODE == kDw ? 2 : 1];
    uint32_t poff[PCOL ? 1 : 2 * NP];     // rows that follow one another: offsets from prow[0], qrow[0]
    uint32_t qoff[MODE == kI8 ? 2 * NQ : 1];
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
            const int tid = here(threadIdx.x), lane = tid & 63, wq = tid >> 7, rr = tid >> 3;
            const int32_t some = n.p0 < a.T ? n.p0 : 0;  // rows past the tile repeat its first
            int32_t in[2 * NQ + 2];
#pragma unroll
            for (int s = 0; s < 2 * NQ + 2; ++s) {
                const int32_t r = n.p0 + (s < 2 * NQ ? s * 32 + rr : wq * 32 * NQ + (s - 2 * NQ) * 64 + lane);
                in[s] = r < n.p1 ? r : some;
            }
#pragma unroll
            for (int s = 0; s < 2 * NQ; ++s) slot[s] = in[s];
#pragma unroll
            for (int u = 0; u < 2; ++u) rows[u] = in[2 * NQ + u];
            if (a.order) {
#pragma unroll
                for (int s = 0; s < 2 * NQ; ++s) slot[s] = a.order[in[s]];
#pragma unroll
                for (int u = 0; u < 2; ++u) rows[u] = a.order[in[2 * NQ + u]];
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
            else if constexpr (MODE == kI8)
                rows[u] = n.p0 + i < n.p1 ? n.p0 + i : -1;
            else
                rows[u] = n.p0 + i < n.p1 && known(rows[u]) ? rows[u] : -1;
        }
    };
    auto set_addresses = [&]() {
        const int rr = here(tid) >> 3;
        if constexpr (MODE == kI8) {
            qrow[0] = a.q + w.p0 * a.qs + rc;
#pragma unroll
            for (int s = 0; s < 2 * NQ; ++s) {
                const int r = s * 32 + rr;
                qoff[s] = w.p0 + r < w.p1 ? (uint32_t)(r * a.qs) : 0u;
            }
        } else if constexpr (!QCOL) {
#pragma unroll
            for (int s = 0; s < 2 * NQ; ++s) {
                int32_t r = known(slot[s]) ? slot[s] : 0;
                if constexpr (MODE == kFwd) r = (int32_t)query_of(a, (uint32_t)r);
                qrow[s] = a.q + (int64_t)r * a.qs + rc;
            }
        }
        const char* pbase = a.p + (RAGGED && w.leaf > 0 ? w.leaf * a.pg : 0);
        if constexpr (!PCOL) {
            prow[0] = pbase + w.j0 * a.ps + rc;
#pragma unroll
            for (int s = 0; s < 2 * NP; ++s) {
                const int r = s * 32 + rr;
                poff[s] = w.j0 + r < a.J ? (uint32_t)(r * a.ps) : 0u;
            }
        } else if constexpr (MODE == kDx) {
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
            if constexpr (!PCOL) {
                *valid = w.red * ELEM - (u * 128 + rc);
                return prow[0] + poff[c] + u * 128;
            } else if constexpr (MODE == kDx) {
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
                if constexpr (MODE == kI8)
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
    v4i pf[2][FP], qf[2][FQ];
    auto load = [&](int u, int c, uint32_t buf) {
        int32_t valid;
        int64_t before;
        const char* src = source(u, c, &valid, &before);
        dma16(valid > 0 ? src : zero, base + buf + c * 4096 + wave * 1024);
    };
    // One half-step: the matrix instructions of fragment set kk; between them the reads of
    // the other set from `buf` and (kk = 1) the loads of step u into the other buffer.
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
        v[0] = a.sw[j];
        v[1] = a.bias ? a.bias[j] : 0.0f;
        v[2] = a.sx[r];
    };
    auto keep_scales = [&](const float(&v)[3]) {
        const int tid = here(threadIdx.x);
        if (tid < 64 * NP) {
            scales[tid] = v[0];
            scales[64 * NP + tid] = v[1];
        }
        if (tid < 64 * NQ) scales[128 * NP + tid] = v[2];
    };

    char* const turn = turns + (OB == 4 ? wave * 16 * kTurnPitch<NP> : 0);

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
        for (; ul < 2; ++ul) {
            if constexpr (MODE == kDw) {
                if (ul == 0)
                    set_rows(0, slot);
                else
                    set_rows(1, slot1);
            }
#pragma unroll
            for (int c = 0; c < 2 * NB; ++c) load(ul, c, ul * BUF);
        }
        us = 1;
        advance_order();
        Tile wc = w;  // what is multiplied
        int32_t uc = 0, rows_c[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) rows_c[u] = rows_l[u];
        clear();
        land<2 * NB>();
#pragma unroll
        for (int x = 0; x < FQ; ++x) qf[0][x] = read_q(x, 0, 0);
#pragma unroll
        for (int x = 0; x < FP; ++x) pf[0][x] = read_p(x, 0, 0);
        for (uint32_t cur = 0;; cur = BUF - cur) {
            float sv[3] = {};
            if constexpr (MODE == kI8) {
                if (uc == 0) load_scales(wc, sv);
            }
            half_step(0, cur, 0);
            land<0>();
            if constexpr (MODE == kI8) {
                if (uc == 0) keep_scales(sv);
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
            half_step(1, BUF - cur, ul++);
            if (++uc < wc.nt) continue;
            if constexpr (NQ * NP > 4) settle();
            out_rows(wc, rows_c);
            store_part<MODE, NQ, NP, OB>(a, acc, scales, turn, rows_c, wc.leaf, wc.j0);
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
            store_part<MODE, NQ, NP, OB>(a, acc, scales, turn, rows, w.leaf, w.j0);
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
// outputs and no others.  HBM-bound (2 or 4 bytes in, 1 out; bfloat16 8192 x 4096: 23 us, 4.3 TB/s; float32
// 40 us, 4.2): one wave per row, no barrier; the row
// is read once and kept in registers up to 8 chunks of 16 bytes a lane.  WHOLE: the rows are
// whole aligned chunks; else chunks at any alignment, the last one short.
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

template <typename T, bool WHOLE>
__global__ __launch_bounds__(256) void i8_quantize_kernel(const T* x, int64_t n, int32_t d, int64_t xs, int8_t* codes,
                                                          float* scale) {
    constexpr int NV = 16 / sizeof(T);
    const int lane = threadIdx.x & 63;
    const int32_t chunks = (d + NV - 1) / NV;
    for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < n; row += (int64_t)gridDim.x * 4) {
        const T* xr = x + row * xs;
        auto fetch = [&](int32_t c) -> v4i {
            const T* p = xr + (int64_t)c * NV;
            if constexpr (WHOLE)
                return *reinterpret_cast<const v4i*>(p);
            else
                return load_chunk<sizeof(T)>(reinterpret_cast<const char*>(p), (int64_t)(d - c * NV) * (int)sizeof(T), (int64_t)c * 16);
        };
        constexpr int KEEP = WHOLE ? 8 : 1;
        v4i keep[KEEP];
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (lane + k * 64 < chunks) keep[k] = fetch(lane + k * 64);
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (lane + k * 64 < chunks) m = fmaxf(m, chunk_max<T>(keep[k]));
        for (int32_t c = lane + KEEP * 64; c < chunks; c += 64) m = fmaxf(m, chunk_max<T>(fetch(c)));
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
        const float s = step_of(m), inv = 1.0f / s;
        if (lane == 0) scale[row] = s;
        auto write = [&](int32_t c, v4i v) {
            int8_t q[NV];
            chunk_codes<T>(v, s, inv, q);
            int8_t* o = codes + row * d + (int64_t)c * NV;
            if (WHOLE || (c + 1) * NV <= d) {
                __builtin_memcpy(o, q, NV);
            } else {
#pragma unroll
                for (int r = 0; r < NV; ++r)
                    if (c * NV + r < d) o[r] = q[r];
            }
        };
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (lane + k * 64 < chunks) write(lane + k * 64, keep[k]);
        for (int32_t c = lane + KEEP * 64; c < chunks; c += 64) write(c, fetch(c));
    }
}

// Few rows: the product is a single pass over the weights.  A workgroup has 16 columns of one matrix and 16 FR
// rows at a time; its eight waves share out the sum, load their pieces of both operands from
// memory into the matrix instruction's layout (lane 16 g + i: 16 bytes of row i), 4 x 64 bytes at once,
// and add up through LDS in a fixed order.  XB = 2 or 4: Q holds tokens of that many bytes an
// element, which every workgroup quantises for itself (as i8_quantize_kernel does, bit for bit).
// HBM-bound in the weights where they are many: 64 slots of 64 leaves, 1536 x 1536, 189 MB of weights
// in 34 us for grouping and product (5.6 TB/s); one token, 1536 -> 4096, 9.5 us a call, a launch's
// latency (7.0 on the GPU; 15.6 with tiles and quantising in a launch of its own).
constexpr int kRowWaves = 8;
template <int MODE, int FR, bool WHOLE, int XB>
__global__ __launch_bounds__(kRowWaves * 64) void prod_rows_kernel(ProdArgs a) {
    constexpr int ELEM = MODE == kI8 ? 1 : 2, U = 4;
    static_assert(XB == 0 || (MODE == kI8 && FR == 1 && WHOLE), "");
    typedef typename Acc<MODE>::type acc_t;
    __shared__ acc_t part[kRowWaves][FR][64];
    __shared__ float most[kRowWaves][16];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, li = lane & 15;
    const int32_t kb = (int32_t)a.red * ELEM, steps = (kb + 63) >> 6;
    const int32_t s0 = steps * wave / kRowWaves, s1 = steps * (wave + 1) / kRowWaves;
    const int32_t j = blockIdx.x * 16 + g * 4;  // this lane's four output columns
    const int32_t leaf = MODE == kI8 ? 0 : blockIdx.y;
    auto put = [&](int32_t row, v4f v) {
        if (a.out_f32) {
            float* o = static_cast<float*>(a.out) + row * a.J + j;
            if (j + 4 <= a.J)
                __builtin_memcpy(o, &v, 16);
            else if (j < a.J)
                store_left<4>(reinterpret_cast<char*>(o), __builtin_bit_cast(v4i, v), (int32_t)a.J - j);
        } else {
            uint16_t* o = static_cast<uint16_t*>(a.out) + row * a.J + j;
            const uint32_t w[2] = {bf16_bits(v[0]) | bf16_bits(v[1]) << 16, bf16_bits(v[2]) | bf16_bits(v[3]) << 16};
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
        for (int32_t p = tid >> 2; p < head + (int32_t)a.T - tail; p += kRowWaves * 16) {
            const int32_t row = slot_of(a, p < head ? p : tail + p - head), c = blockIdx.x * 16 + (tid & 3) * 4;
            if (row < 0 || c >= a.J) continue;
            const int32_t left = (int32_t)a.J - c, ob = a.out_f32 ? 4 : 2;
            char* o = static_cast<char*>(a.out) + (row * a.J + c) * ob;
            for (int32_t e = 0; e < (left < 4 ? left : 4) * ob; e += 2) *reinterpret_cast<uint16_t*>(o + e) = 0;
        }
        return;
    }
    const int32_t col = blockIdx.x * 16 + li < a.J ? blockIdx.x * 16 + li : (int32_t)a.J - 1;
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
        v4i pv[U], qv[U][FR], xv[XB > 0 ? U : 1][XB > 0 ? XB : 1];
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
        acc_t acc[FR];
#pragma unroll
        for (int f = 0; f < FR; ++f) acc[f] = acc_t{0, 0, 0, 0};
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
                    for (int f = 0; f < FR; ++f) acc[f] = mma<MODE>(pv[u], qv[u][f], acc[f]);
                }
        }
#pragma unroll
        for (int f = 0; f < FR; ++f) part[wave][f][lane] = acc[f];
        __syncthreads();
#pragma unroll
        for (int f = 0; f < FR; ++f)
            if (wave == f && out_row[f] >= 0) {
                acc_t t = part[0][f][lane];
#pragma unroll
                for (int w = 1; w < kRowWaves; ++w) t += part[w][f][lane];
                v4f v;
                if constexpr (MODE == kI8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = (float)t[e] * sx * sw[e];
                        if (a.bias) v[e] += bias[e];
                    }
                } else {
                    v = t;
                }
                put(out_row[f], v);
            }
        if (p + (int32_t)gridDim.z * 16 * FR < p1) __syncthreads();
    }
}

// Sum of each row's `fan` float32 partial gradients, rounded once.  HBM-bound (8192 rows x 2 x 1536 to float32:
// 22 us, 6.9 TB/s, part of it from the last-level cache); four columns a thread
// (cols % 4 == 0: the partial rows are 16-byte aligned; else one).
template <int N>
__global__ __launch_bounds__(256) void fan_sum_kernel(const float* part, int64_t rows, int32_t fan, int64_t cols,
                                                      void* out, int32_t out_f32) {
    const int64_t per = cols / N, total = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per, c = (i - r * per) * N;
        float s[N] = {};
        for (int32_t f = 0; f < fan; ++f) {
            float v[N];
            __builtin_memcpy(v, part + (r * fan + f) * cols + c, 4 * N);
#pragma unroll
            for (int e = 0; e < N; ++e) s[e] += v[e];
        }
        if (out_f32) {
            __builtin_memcpy(static_cast<float*>(out) + r * cols + c, s, 4 * N);
        } else {
            uint16_t b[N];
#pragma unroll
            for (int e = 0; e < N; ++e) b[e] = (uint16_t)bf16_bits(s[e]);
            __builtin_memcpy(static_cast<uint16_t*>(out) + r * cols + c, b, 2 * N);
        }
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
    if (MODE == kI8) return (a.T + TQ - 1) / TQ;
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

template <int MODE, int NQ, int NP, bool DMA>
hipError_t launch_tiles(const ProdArgs& a, hipStream_t stream) {
    constexpr int TQ = NQ * 64, TP = NP * 64;
    const int64_t np = (a.J + TP - 1) / TP, each = row_tiles<MODE>(a, TQ, true) * np;
    const int64_t resident = kCUs * (NQ * NP > 4 ? 1 : 2);
    int64_t wgs = (each + 7) / 8 * 8;
    if (MODE == kDw) {  // a workgroup for each tile: they are of unequal length, and start as others end
        const int64_t leaf = (a.I + TQ - 1) / TQ * np;
        if (leaf >= 8) wgs = (leaf + 7) / 8 * 8 * a.L;
    }
    if ((MODE != kDw || wgs * kNT > kMaxGridItems) && wgs > resident) wgs = resident;
    const dim3 grid((uint32_t)wgs);
    if (a.out_f32)
        hipLaunchKernelGGL((prod_tile_kernel<MODE, NQ, NP, 4, DMA>), grid, dim3(kNT), 0, stream, a);
    else
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
    if constexpr (XB == 0) {
        if (!whole) {
            hipLaunchKernelGGL((prod_rows_kernel<MODE, FR, false, 0>), grid, dim3(kRowWaves * 64), 0, stream, a);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((prod_rows_kernel<MODE, FR, true, XB>), grid, dim3(kRowWaves * 64), 0, stream, a);
    return hipGetLastError();
}

template <int MODE>
hipError_t launch_prod(ProdArgs a, int32_t fan, hipStream_t stream) {
    const int e = MODE == kI8 ? 1 : 2;
    bool whole;
    if (MODE == kDw)
        whole = chunked(a.q, a.qs, a.I * e) && chunked(a.p, a.ps, a.J * e);
    else if (MODE == kDx)
        whole = chunked(a.q, a.qs, a.red * e) && chunked(a.p, a.ps, a.J * e);
    else
        whole = chunked(a.q, a.qs, a.red * e) && chunked(a.p, a.ps, 0);
    // ceil(2^(31 + l) / fan) with l = ceil(log2 fan) divides every slot below 2^31 exactly
    int l = 0;
    while (((int64_t)1 << l) < fan) ++l;
    a.fan_shift = 31 + l;
    a.fan_mul = (uint32_t)((((uint64_t)1 << (31 + l)) + fan - 1) / fan);
    const int64_t pitch = a.J * (a.out_f32 ? 4 : 2);
    a.bypass = MODE != kFwd && ((reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)pitch) & 63) == 0;
    if constexpr (MODE == kI8 || MODE == kFwd) {
        switch (row_fragments<MODE>(a)) {
            case 1: return launch_rows<MODE, 1>(a, whole, stream);
            case 2: return launch_rows<MODE, 2>(a, whole, stream);
            case 4: return launch_rows<MODE, 4>(a, whole, stream);
        }
    }
    if (!whole) return launch_tiles<MODE, 2, 2, false>(a, stream);
    if constexpr (MODE == kDw) {
        return launch_tiles<MODE, 2, 2, true>(a, stream);
    } else {
        switch (tile_shape<MODE>(a)) {
            case 4: return launch_tiles<MODE, 4, 4, true>(a, stream);
            case 3: return launch_tiles<MODE, 3, 4, true>(a, stream);
            default: return launch_tiles<MODE, 2, 2, true>(a, stream);
        }
    }
}

}  // namespace

hipError_t launch_i8_quantize(const void* x, int32_t dtype, int64_t n, int32_t d, int64_t xs, int8_t* codes,
                              float* scale, hipStream_t stream) {
    const int64_t e = dtype == AH_F32 ? 4 : 2;
    const dim3 grid((uint32_t)(n < (1 << 22) ? (n + 3) / 4 : 1 << 20));
    const bool whole = chunked(x, xs * e, d * e);
    auto go = [&](auto kernel, auto* rows) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, rows, n, d, xs, codes, scale);
    };
    if (dtype == AH_F32)
        go(whole ? i8_quantize_kernel<float, true> : i8_quantize_kernel<float, false>, static_cast<const float*>(x));
    else
        go(whole ? i8_quantize_kernel<uint16_t, true> : i8_quantize_kernel<uint16_t, false>,
           static_cast<const uint16_t*>(x));
    return hipGetLastError();
}

static ProdArgs i8_args(const int8_t* x8, const float* xs, int64_t m, const int8_t* w8, const float* ws, int64_t n,
                        int32_t k, const float* bias, void* out, int32_t out_dtype) {
    ProdArgs a{};
    a.q = reinterpret_cast<const char*>(x8);
    a.p = reinterpret_cast<const char*>(w8);
    a.qs = a.ps = k;
    a.T = a.I = m;
    a.J = n;
    a.red = k;
    a.out = out;
    a.out_f32 = out_dtype == AH_F32;
    a.sx = xs;
    a.sw = ws;
    a.bias = bias;
    return a;
}

hipError_t launch_i8_matmul(const int8_t* x8, const float* xs, int64_t m, const int8_t* w8, const float* ws, int64_t n,
                            int32_t k, const float* bias, void* out, int32_t out_dtype, hipStream_t stream) {
    return launch_prod<kI8>(i8_args(x8, xs, m, w8, ws, n, k, bias, out, out_dtype), 1, stream);
}

// Workspace: the tokens' codes (rows of k bytes, the block rounded up to 16) and their steps.
static size_t code_bytes(int64_t m, int32_t k) { return ((size_t)m * k + 15) / 16 * 16; }
size_t i8_linear_workspace_bytes(int64_t m, int32_t k) { return code_bytes(m, k) + (size_t)m * sizeof(float); }

hipError_t launch_i8_linear(const void* x, int32_t dtype, int64_t m, int32_t k, int64_t xs, const int8_t* w8,
                            const float* ws, int64_t n, const float* bias, void* out, int32_t out_dtype, void* work,
                            hipStream_t stream) {
    const int64_t bytes = dtype == AH_F32 ? 4 : 2;
    if (m <= 16 && rows_launchable(n) && chunked(x, xs * bytes, k) && chunked(w8, k, 0)) {
        ProdArgs a = i8_args(static_cast<const int8_t*>(x), nullptr, m, w8, ws, n, k, bias, out, out_dtype);
        a.qs = xs * bytes;
        return dtype == AH_F32 ? launch_rows<kI8, 1, 4>(a, true, stream) : launch_rows<kI8, 1, 2>(a, true, stream);
    }
    int8_t* codes = static_cast<int8_t*>(work);
    float* scale = reinterpret_cast<float*>(codes + code_bytes(m, k));
    const hipError_t e = launch_i8_quantize(x, dtype, m, k, xs, codes, scale, stream);
    if (e != hipSuccess) return e;
    return launch_i8_matmul(codes, scale, m, w8, ws, n, k, bias, out, out_dtype, stream);
}

hipError_t launch_grouped(const GroupedProblem& g, void* out, int32_t out_dtype, hipStream_t stream) {
    ProdArgs a{};
    a.q = static_cast<const char*>(g.x);
    a.qs = g.x_stride * 2;
    a.p = static_cast<const char*>(g.w);
    a.ps = (int64_t)g.k * 2;
    a.pg = (int64_t)g.n * g.k * 2;
    a.off = g.offsets;
    a.order = g.order;
    a.T = a.I = g.slots;
    a.L = g.L;
    a.J = g.n;
    a.red = g.k;
    a.out = out;
    a.out_f32 = out_dtype == AH_F32;
    return launch_prod<kFwd>(a, g.fan, stream);
}

size_t grouped_dx_workspace_bytes(int64_t slots, int32_t k, int32_t fan) {
    return fan > 1 ? (size_t)slots * k * sizeof(float) : 0;
}

hipError_t launch_grouped_dx(const GroupedProblem& g, void* out, int32_t out_dtype, void* ws, hipStream_t stream) {
    ProdArgs a{};
    a.q = static_cast<const char*>(g.dy);
    a.qs = g.dy_stride * 2;
    a.p = static_cast<const char*>(g.w);
    a.ps = (int64_t)g.k * 2;
    a.pg = (int64_t)g.n * g.k * 2;
    a.off = g.offsets;
    a.order = g.order;
    a.T = a.I = g.slots;
    a.L = g.L;
    a.J = g.k;
    a.red = g.n;
    a.out = g.fan > 1 ? ws : out;
    a.out_f32 = g.fan > 1 || out_dtype == AH_F32;
    hipError_t e = launch_prod<kDx>(a, g.fan, stream);
    if (e != hipSuccess || g.fan == 1) return e;
    const int64_t rows = g.slots / g.fan, n = g.k % 4 == 0 ? 4 : 1, wgs = (rows * g.k / n + 255) / 256;
    const dim3 grid((uint32_t)(wgs < 16384 ? wgs : 16384));
    const float* part = static_cast<const float*>(ws);
    if (n == 4)
        hipLaunchKernelGGL(fan_sum_kernel<4>, grid, dim3(256), 0, stream, part, rows, g.fan, (int64_t)g.k, out,
                           out_dtype == AH_F32);
    else
        hipLaunchKernelGGL(fan_sum_kernel<1>, grid, dim3(256), 0, stream, part, rows, g.fan, (int64_t)g.k, out,
                           out_dtype == AH_F32);
    return hipGetLastError();
}

hipError_t launch_grouped_dw(const GroupedProblem& g, void* out, int32_t out_dtype, hipStream_t stream) {
    ProdArgs a{};
    a.q = static_cast<const char*>(g.dy);
    a.qs = g.dy_stride * 2;
    a.p = static_cast<const char*>(g.x);
    a.ps = g.x_stride * 2;
    a.off = g.offsets;
    a.order = g.slots > 0 ? g.order : nullptr;
    a.T = g.slots;
    a.I = g.n;
    a.L = g.L;
    a.J = g.k;
    a.out = out;
    a.out_f32 = out_dtype == AH_F32;
    return launch_prod<kDw>(a, g.fan, stream);
}

}  // namespace ah
