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
// Tiles.  One step of the sum is 128 bytes of t (128 int8 or 64 bfloat16 values),
// and every operand's step is cut into half-tiles of 16 KB: 128 rows x 128 bytes
// ("row" operands) or 64 memory rows x 256 bytes ("by column").  Global memory goes
// straight to LDS (16 bytes a lane); that write is linear in the lane, so
// the swizzle that keeps the reads free of bank conflicts is applied to the
// source address: a row operand's 16-byte chunk c of row r lies at c ^ (r & 7), a
// by-column operand's 32-byte granule c of memory row r at c ^ (r & 3 | (r >> 3 & 1) << 2),
// which puts the eight rows that half a wave reads at once into eight different
// granules.  The matrix instruction takes P as its A operand, so that a lane ends
// with four consecutive output columns of one row.
#include "ah_device.hpp"
#include "ah_kernels.hpp"
#include "../../include/ah.h"

namespace ah {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef int v2i __attribute__((ext_vector_type(2)));

enum { kI8 = 0, kFwd = 1, kDx = 2, kDw = 3 };

constexpr int kNT = 512;         // threads: 2 wave rows x 4 wave columns
constexpr int kHalf = 16384;     // bytes of a half-tile
constexpr int kFQ = 4, kFP = 2;  // 16-row fragments of a half-tile that one wave reads, row and column side

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
    int32_t L, fan;
    int64_t I, J;          // output rows of one matrix (dw: n; else T) and columns
    int64_t red;           // summed elements (dw: unused, the leaf's rows)
    void* out;
    int32_t out_f32;
    const float *sx, *sw, *bias;  // int8
};

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}
__device__ __forceinline__ void dma16(const char* src, char* lds) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                     (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}
template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wg_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

// Fragments of one half-tile, both 64-byte steps: f[x][kk].  The reads wait in
// their own block: a separate wait could be passed by a use of the registers.
template <int F>
__device__ __forceinline__ void read_rows(v4i (&f)[F][2], uint32_t a0, uint32_t a1) {
    if constexpr (F == 4) {
        asm volatile(
            "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\t"
            "ds_read_b128 %2, %8 offset:2048\n\tds_read_b128 %3, %9 offset:2048\n\t"
            "ds_read_b128 %4, %8 offset:4096\n\tds_read_b128 %5, %9 offset:4096\n\t"
            "ds_read_b128 %6, %8 offset:6144\n\tds_read_b128 %7, %9 offset:6144\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(f[0][0]), "=&v"(f[0][1]), "=&v"(f[1][0]), "=&v"(f[1][1]), "=&v"(f[2][0]), "=&v"(f[2][1]),
              "=&v"(f[3][0]), "=&v"(f[3][1])
            : "v"(a0), "v"(a1)
            : "memory");
    } else {
        asm volatile(
            "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\t"
            "ds_read_b128 %2, %4 offset:2048\n\tds_read_b128 %3, %5 offset:2048\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(f[0][0]), "=&v"(f[0][1]), "=&v"(f[1][0]), "=&v"(f[1][1])
            : "v"(a0), "v"(a1)
            : "memory");
    }
}
__device__ __forceinline__ v4i join(v2i a, v2i b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3); }
// By-column: fragment x at a[x]; its summed rows g * 8 .. g * 8 + 7 (g = lane / 16) are two transposed reads.
template <int F>
__device__ __forceinline__ void read_cols(v4i (&f)[F][2], const uint32_t (&a)[F]) {
    v2i r[F][4];
    if constexpr (F == 4) {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %16\n\tds_read_b64_tr_b16 %1, %16 offset:1024\n\t"
            "ds_read_b64_tr_b16 %2, %16 offset:8192\n\tds_read_b64_tr_b16 %3, %16 offset:9216\n\t"
            "ds_read_b64_tr_b16 %4, %17\n\tds_read_b64_tr_b16 %5, %17 offset:1024\n\t"
            "ds_read_b64_tr_b16 %6, %17 offset:8192\n\tds_read_b64_tr_b16 %7, %17 offset:9216\n\t"
            "ds_read_b64_tr_b16 %8, %18\n\tds_read_b64_tr_b16 %9, %18 offset:1024\n\t"
            "ds_read_b64_tr_b16 %10, %18 offset:8192\n\tds_read_b64_tr_b16 %11, %18 offset:9216\n\t"
            "ds_read_b64_tr_b16 %12, %19\n\tds_read_b64_tr_b16 %13, %19 offset:1024\n\t"
            "ds_read_b64_tr_b16 %14, %19 offset:8192\n\tds_read_b64_tr_b16 %15, %19 offset:9216\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[0][2]), "=&v"(r[0][3]), "=&v"(r[1][0]), "=&v"(r[1][1]),
              "=&v"(r[1][2]), "=&v"(r[1][3]), "=&v"(r[2][0]), "=&v"(r[2][1]), "=&v"(r[2][2]), "=&v"(r[2][3]),
              "=&v"(r[3][0]), "=&v"(r[3][1]), "=&v"(r[3][2]), "=&v"(r[3][3])
            : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3])
            : "memory");
    } else {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %8\n\tds_read_b64_tr_b16 %1, %8 offset:1024\n\t"
            "ds_read_b64_tr_b16 %2, %8 offset:8192\n\tds_read_b64_tr_b16 %3, %8 offset:9216\n\t"
            "ds_read_b64_tr_b16 %4, %9\n\tds_read_b64_tr_b16 %5, %9 offset:1024\n\t"
            "ds_read_b64_tr_b16 %6, %9 offset:8192\n\tds_read_b64_tr_b16 %7, %9 offset:9216\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[0][2]), "=&v"(r[0][3]), "=&v"(r[1][0]), "=&v"(r[1][1]),
              "=&v"(r[1][2]), "=&v"(r[1][3])
            : "v"(a[0]), "v"(a[1])
            : "memory");
    }
#pragma unroll
    for (int x = 0; x < F; ++x) {
        f[x][0] = join(r[x][0], r[x][1]);
        f[x][1] = join(r[x][2], r[x][3]);
    }
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

// 16 bytes of which the first `valid` (<= 0: none) exist; ELEM bytes an element.
template <int ELEM>
__device__ __forceinline__ v4i load_chunk(const char* src, int64_t valid) {
    v4i r = {0, 0, 0, 0};
    if (valid >= 16) {
        __builtin_memcpy(&r, src, 16);
    } else if (valid > 0) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t v = 0;
#pragma unroll
            for (int b = 0; b < 4; b += ELEM) {
                if (4 * w + b < valid) {
                    if constexpr (ELEM == 1) {
                        v |= (uint32_t)(uint8_t)src[4 * w + b] << (8 * b);
                    } else {
                        uint16_t u;
                        __builtin_memcpy(&u, src + 4 * w + b, 2);
                        v |= (uint32_t)u << (8 * b);
                    }
                }
            }
            r[w] = (int)v;
        }
    }
    return r;
}

__device__ __forceinline__ uint32_t bf16_bits(float f) {  // round to nearest even; NaN stays NaN
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f);
}
// Up to four consecutive outputs, `left` of which exist, at any element alignment.
__device__ __forceinline__ void store4(void* out, int32_t f32, int64_t at, v4f v, int64_t left) {
    if (f32) {
        float* o = static_cast<float*>(out) + at;
        if (left >= 4) {
            __builtin_memcpy(o, &v, 16);
        } else {
            for (int r = 0; r < left; ++r) o[r] = v[r];
        }
    } else {
        uint16_t* o = static_cast<uint16_t*>(out) + at;
        uint32_t w[2] = {bf16_bits(v[0]) | bf16_bits(v[1]) << 16, bf16_bits(v[2]) | bf16_bits(v[3]) << 16};
        if (left >= 4) {
            __builtin_memcpy(o, w, 8);
        } else {
            for (int r = 0; r < left; ++r) o[r] = (uint16_t)(w[r >> 1] >> (16 * (r & 1)));
        }
    }
}

struct Where {
    int32_t leaf;   // -1: rows of no leaf (their outputs are zero)
    int32_t qt;     // row tile inside the matrix (int8, dw)
    int64_t p0, p1; // grouped rows of this tile, forward and dx (dw: the leaf's rows)
    int64_t tp;     // column tile
};

// Tile of a workgroup.  Consecutive workgroups go to the eight XCDs in turn, so
// XCD x is given the x-th eighth of the tiles (their operands then share its L2),
// and inside it eight row tiles are walked for each column tile.
__device__ __forceinline__ int64_t xcd_tile(int64_t total) {
    const int64_t per = (total + 7) >> 3, i = (int64_t)blockIdx.x >> 3;
    const int64_t t = (int64_t)(blockIdx.x & 7) * per + i;
    return i < per && t < total ? t : -1;
}
__device__ __forceinline__ void walk(int64_t t, int64_t nq, int64_t np, int64_t* tq, int64_t* tp) {
    constexpr int G = 8;
    const int64_t band = t / (G * np), r = t - band * G * np;
    const int64_t h = nq - band * G < G ? nq - band * G : G;
    *tp = r / h;
    *tq = band * G + r % h;
}

struct LocateShared {
    int64_t wave_sum[kNT / 64];
    Where w;
};
__device__ __forceinline__ int64_t leaf_start(const ProdArgs& a, int32_t l) {  // inside [0, T] whatever the array holds
    const int64_t o = a.off[l];
    return o < 0 ? 0 : o > a.T ? a.T : o;
}
// Rows of entry e: a leaf, or (L, L + 1) the rows after the last and before the first leaf.
__device__ __forceinline__ void entry_rows(const ProdArgs& a, int32_t e, int64_t* b, int64_t* n) {
    *b = e <= a.L ? leaf_start(a, e) : 0;
    *n = (e < a.L ? leaf_start(a, e + 1) : e == a.L ? a.T : leaf_start(a, 0)) - *b;
    if (*n < 0) *n = 0;
}
// The leaf and rows of this workgroup's tile, from the leaf starts on the device:
// a prefix sum of the leaves' row tiles, one entry or a run of them per thread.
template <int TQ>
__device__ bool locate(const ProdArgs& a, int64_t np, LocateShared& sh, Where* out) {
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int32_t E = a.L + 2, run = (E + kNT - 1) / kNT;
    int64_t sum = 0;
    for (int32_t e = tid * run; e < E && e < (tid + 1) * run; ++e) {
        int64_t b, n;
        entry_rows(a, e, &b, &n);
        sum += (n + TQ - 1) / TQ;
    }
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t v = __shfl_up(incl, o, 64);
        if (lane >= o) incl += v;
    }
    if (lane == 63) sh.wave_sum[wave] = incl;
    if (tid == 0) sh.w.leaf = -2;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kNT / 64; ++w) {
        const int64_t s = sh.wave_sum[w];
        if (w < wave) incl += s;
        total += s;
    }
    const int64_t t = xcd_tile(total * np);
    if (t < 0) return false;
    int64_t tq, tp;
    walk(t, total, np, &tq, &tp);
    int64_t at = incl - sum;
    if (tq >= at && tq < incl) {
        for (int32_t e = tid * run; e < E && e < (tid + 1) * run; ++e) {
            int64_t b, n;
            entry_rows(a, e, &b, &n);
            const int64_t k = (n + TQ - 1) / TQ;
            if (tq < at + k) {
                sh.w.leaf = e < a.L ? e : -1;
                sh.w.p0 = b + (tq - at) * TQ;
                sh.w.p1 = sh.w.p0 + TQ < b + n ? sh.w.p0 + TQ : b + n;
                sh.w.tp = tp;
                break;
            }
            at += k;
        }
    }
    __syncthreads();
    *out = sh.w;
    __syncthreads();
    return out->leaf != -2;
}

// Slot of grouped row p, or -1 if the order holds none there.
__device__ __forceinline__ int64_t slot_of(const ProdArgs& a, int64_t p) {
    if (!a.order) return p;
    const int64_t s = a.order[p];
    return s >= 0 && s < a.T ? s : -1;
}

// Tile of HQ x HP half-tiles.  DMA: operands are 16-byte aligned with whole chunks;
// otherwise chunks go through registers, where a chunk's missing elements become zero.
template <int MODE, int HQ, int HP, bool DMA>
__global__ __launch_bounds__(kNT, HQ* HP >= 4 ? 2 : 4) void prod_tile_kernel(ProdArgs a) {
    constexpr int ELEM = MODE == kI8 ? 1 : 2;
    constexpr bool QCOL = MODE == kDw, PCOL = MODE >= kDx;
    constexpr int TQ = HQ * 128, TP = HP * 128, STEP = 128 / ELEM;
    constexpr int BUF = (HQ + HP) * kHalf;
    __shared__ __align__(1024) char lds[2 * BUF];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wq = wave >> 2, wp = wave & 3, g = lane >> 4, li = lane & 15;
    const int64_t np = (a.J + TP - 1) / TP;

    Where w;
    if constexpr (MODE == kFwd || MODE == kDx) {
        static_assert(sizeof(LocateShared) <= sizeof(lds), "");
        if (!locate<TQ>(a, np, *reinterpret_cast<LocateShared*>(lds), &w)) return;
    } else {
        const int64_t nq = (a.I + TQ - 1) / TQ;
        const int64_t t = xcd_tile(nq * np * (MODE == kDw ? a.L : 1));
        if (t < 0) return;
        w.leaf = (int32_t)(t / (nq * np));
        int64_t tq, tp;
        walk(t - w.leaf * nq * np, nq, np, &tq, &tp);
        w.qt = (int32_t)tq;
        w.tp = tp;
        if constexpr (MODE == kDw) {
            w.p0 = leaf_start(a, w.leaf);
            w.p1 = leaf_start(a, w.leaf + 1);
        } else {
            w.p0 = tq * TQ;
            w.p1 = w.p0 + TQ < a.T ? w.p0 + TQ : a.T;
        }
    }
    const int64_t j0 = w.tp * TP;
    const int64_t red = MODE == kDw ? (w.p1 > w.p0 ? w.p1 - w.p0 : 0) : w.leaf < 0 ? 0 : a.red;
    const int nt = (int)((red + STEP - 1) / STEP);
    const char* const zero = reinterpret_cast<const char*>(&zero_chunk);

    // this thread's 16-byte chunks: rows 64 s + tid / 8 of a row operand's half-tile,
    // memory rows 32 s + tid / 16 of a by-column one (s = 0, 1)
    const int rr = tid >> 3, rc = ((tid & 7) ^ (rr & 7)) * 16;
    const int cr = tid >> 4, cf = (cr & 3) | ((cr >> 3) & 1) << 2;
    const int cc = ((((tid & 15) >> 1) ^ cf) << 1 | (tid & 1)) * 16;

    const char* qrow[QCOL ? 1 : HQ][2];
    const char* prow[PCOL ? 1 : HP][2];
    const char* pbase = a.p + (MODE == kFwd || MODE == kDx ? (w.leaf < 0 ? 0 : w.leaf) * a.pg : 0);
    if constexpr (!QCOL) {
#pragma unroll
        for (int h = 0; h < HQ; ++h)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                int64_t r = w.p0 + h * 128 + s * 64 + rr;
                if (r >= w.p1) r = w.p0;  // rows past the tile repeat its first; their outputs are not written
                if constexpr (MODE != kI8) {
                    r = slot_of(a, r);
                    if (r < 0) r = 0;
                    if constexpr (MODE == kFwd) r = (uint32_t)r / (uint32_t)a.fan;
                }
                qrow[h][s] = a.q + r * a.qs;
            }
    }
    if constexpr (!PCOL) {
#pragma unroll
        for (int h = 0; h < HP; ++h)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                int64_t r = j0 + h * 128 + s * 64 + rr;
                if (r >= a.J) r = j0;
                prow[h][s] = pbase + r * a.ps;
            }
    }

    // Chunk s of half-tile h at sum step t: its address, and in *valid the bytes of it that exist.
    const int64_t rend = red * ELEM;
    auto q_src = [&](int t, int h, int s, int64_t* valid) -> const char* {
        if constexpr (!QCOL) {
            const int64_t o = (int64_t)t * 128 + rc;
            *valid = rend - o;
            return qrow[h][s] + o;
        } else {
            const int64_t o = (int64_t)w.qt * (TQ * 2) + h * 256 + cc;
            const int64_t p = w.p0 + (int64_t)t * STEP + s * 32 + cr;
            const int64_t r = p < w.p1 ? slot_of(a, p) : -1;
            *valid = r < 0 ? 0 : a.I * 2 - o;
            return a.q + r * a.qs + o;
        }
    };
    auto p_src = [&](int t, int h, int s, int64_t* valid) -> const char* {
        if constexpr (!PCOL) {
            const int64_t o = (int64_t)t * 128 + rc;
            *valid = rend - o;
            return prow[h][s] + o;
        } else if constexpr (MODE == kDx) {
            const int64_t o = j0 * 2 + h * 256 + cc, r = (int64_t)t * STEP + s * 32 + cr;
            *valid = r < red ? a.J * 2 - o : 0;
            return pbase + r * a.ps + o;
        } else {
            const int64_t o = j0 * 2 + h * 256 + cc;
            const int64_t p = w.p0 + (int64_t)t * STEP + s * 32 + cr;
            const int64_t r = p < w.p1 ? slot_of(a, p) : -1;
            *valid = r < 0 ? 0 : a.J * 2 - o;
            return a.p + (int64_t)((uint32_t)r / (uint32_t)a.fan) * a.ps + o;
        }
    };

    // fragment addresses inside a buffer (column side first, then row side)
    const uint32_t base = lds_addr(lds);
    uint32_t pa[PCOL ? kFP : 2], qa[QCOL ? kFQ : 2];
    const int fi = (li >> 2) | (g & 1) << 2;
    if constexpr (PCOL) {
#pragma unroll
        for (int x = 0; x < kFP; ++x) pa[x] = base + (g * 8 + (li >> 2)) * 256 + ((wp * kFP + x) ^ fi) * 32 + (li & 3) * 8;
    } else {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) pa[kk] = base + (wp * kFP * 16 + li) * 128 + (((kk * 4 + g) ^ (li & 7)) * 16);
    }
    if constexpr (QCOL) {
#pragma unroll
        for (int x = 0; x < kFQ; ++x)
            qa[x] = base + HP * kHalf + (g * 8 + (li >> 2)) * 256 + ((wq * kFQ + x) ^ fi) * 32 + (li & 3) * 8;
    } else {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
            qa[kk] = base + HP * kHalf + (wq * kFQ * 16 + li) * 128 + (((kk * 4 + g) ^ (li & 7)) * 16);
    }

    typedef typename Acc<MODE>::type acc_t;
    acc_t acc[HQ][HP][kFQ][kFP];
#pragma unroll
    for (int x = 0; x < HQ * HP * kFQ * kFP; ++x) (&acc[0][0][0][0])[x] = acc_t{0, 0, 0, 0};

    v4i stage[DMA ? 1 : 2 * (HQ + HP)];
    auto fetch = [&](int t, int buf) {
        char* l = lds + buf * BUF + wave * 1024;
#pragma unroll
        for (int h = 0; h < HP + HQ; ++h)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                int64_t valid;
                const char* src = h < HP ? p_src(t, h, s, &valid) : q_src(t, h - HP, s, &valid);
                if constexpr (DMA)
                    dma16(valid > 0 ? src : zero, l + h * kHalf + s * 8192);
                else
                    stage[2 * h + s] = load_chunk<ELEM>(src, valid);
            }
    };
    auto compute = [&](int buf) {
        const uint32_t b = buf * BUF;
        v4i pf[HP][kFP][2], qf[kFQ][2];
#pragma unroll
        for (int h = 0; h < HP; ++h) {
            if constexpr (PCOL) {
                uint32_t ad[kFP];
#pragma unroll
                for (int x = 0; x < kFP; ++x) ad[x] = pa[x] + b + h * kHalf;
                read_cols<kFP>(pf[h], ad);
            } else {
                read_rows<kFP>(pf[h], pa[0] + b + h * kHalf, pa[1] + b + h * kHalf);
            }
        }
#pragma unroll
        for (int h = 0; h < HQ; ++h) {
            if constexpr (QCOL) {
                uint32_t ad[kFQ];
#pragma unroll
                for (int x = 0; x < kFQ; ++x) ad[x] = qa[x] + b + h * kHalf;
                read_cols<kFQ>(qf, ad);
            } else {
                read_rows<kFQ>(qf, qa[0] + b + h * kHalf, qa[1] + b + h * kHalf);
            }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int hp = 0; hp < HP; ++hp)
#pragma unroll
                    for (int x = 0; x < kFQ; ++x)
#pragma unroll
                        for (int y = 0; y < kFP; ++y)
                            acc[h][hp][x][y] = mma<MODE>(pf[hp][y][kk], qf[x][kk], acc[h][hp][x][y]);
        }
    };

    if constexpr (DMA) {
        if (nt > 0) fetch(0, 0);
        for (int t = 0; t < nt; ++t) {
            wait_vm<0>();  // step t has landed, and every wave is done with the other buffer
            wg_barrier();
            if (t + 1 < nt) fetch(t + 1, (t + 1) & 1);
            compute(t & 1);
        }
    } else {
        if (nt > 0) fetch(0, 0);
        for (int t = 0; t < nt; ++t) {
            __syncthreads();
#pragma unroll
            for (int h = 0; h < HP + HQ; ++h)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    *reinterpret_cast<v4i*>(lds + h * kHalf + s * 8192 + tid * 16) = stage[2 * h + s];
            __syncthreads();
            if (t + 1 < nt) fetch(t + 1, 0);
            compute(0);
        }
    }

#pragma unroll
    for (int h = 0; h < HQ; ++h)
#pragma unroll
        for (int x = 0; x < kFQ; ++x) {
            const int i = h * 128 + wq * 64 + x * 16 + li;
            int64_t row;
            float sx = 0.0f;
            if constexpr (MODE == kDw) {
                row = (int64_t)w.qt * TQ + i;
                if (row >= a.I) continue;
                row += w.leaf * a.I;
            } else {
                row = w.p0 + i;
                if (row >= w.p1) continue;
                if constexpr (MODE == kI8) {
                    sx = a.sx[row];
                } else {
                    row = slot_of(a, row);
                    if (row < 0) continue;
                }
            }
#pragma unroll
            for (int hp = 0; hp < HP; ++hp)
#pragma unroll
                for (int y = 0; y < kFP; ++y) {
                    const int64_t j = j0 + hp * 128 + wp * 32 + y * 16 + g * 4;
                    if (j >= a.J) continue;
                    v4f v;
                    if constexpr (MODE == kI8) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int64_t jr = j + r < a.J ? j + r : a.J - 1;
                            v[r] = (float)acc[h][hp][x][y][r] * sx * a.sw[jr];
                            if (a.bias) v[r] += a.bias[jr];
                        }
                    } else {
                        v = acc[h][hp][x][y];
                    }
                    store4(a.out, a.out_f32, row * a.J + j, v, a.J - j);
                }
        }
}

// Tokens to int8 codes: step = max |x| / 127 (float32), code = rint(x / step).
// One workgroup per row; a row with a NaN or an infinity gets step NaN and zero
// codes, so that it spoils its own outputs and no others.
template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    if constexpr (sizeof(T) == 4)
        return __builtin_bit_cast(float, v);
    else
        return __uint_as_float((uint32_t)v << 16);
}
template <typename T>
__global__ __launch_bounds__(256) void i8_quantize_kernel(const T* x, int64_t n, int32_t d, int64_t xs, int8_t* codes,
                                                          float* scale) {
    __shared__ float red[4];
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        const T* xr = x + row * xs;
        float m = 0.0f;
        for (int32_t j = threadIdx.x; j < d; j += 256) {
            const float v = fabsf(to_f32(xr[j]));
            m = v < INFINITY ? fmaxf(m, v) : NAN;
            if (!(v < INFINITY)) break;
        }
        bool bad = !(m < INFINITY);
        m = bad ? 0.0f : m;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
        const int any = __syncthreads_or(bad);
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
        __syncthreads();
        const float s = any ? NAN : fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])) / 127.0f;
        if (threadIdx.x == 0) scale[row] = s;
        for (int32_t j = threadIdx.x; j < d; j += 256) {
            const float q = s > 0.0f ? rintf(to_f32(xr[j]) / s) : 0.0f;
            codes[row * d + j] = (int8_t)(int)fminf(fmaxf(q, -127.0f), 127.0f);
        }
        __syncthreads();
    }
}

// Sum of each row's `fan` float32 partial gradients, rounded once.
__global__ __launch_bounds__(256) void fan_sum_kernel(const float* part, int64_t rows, int32_t fan, int64_t cols,
                                                      void* out, int32_t out_f32) {
    const int64_t total = rows * cols;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / cols, c = i - r * cols;
        float s = 0.0f;
        for (int32_t f = 0; f < fan; ++f) s += part[(r * fan + f) * cols + c];
        if (out_f32)
            static_cast<float*>(out)[i] = s;
        else
            static_cast<uint16_t*>(out)[i] = (uint16_t)bf16_bits(s);
    }
}

inline bool chunked(const void* p, int64_t stride_bytes, int64_t width_bytes) {
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride_bytes | (uintptr_t)width_bytes) & 15) == 0;
}

template <int MODE, bool DMA>
hipError_t launch_tiles(const ProdArgs& a, hipStream_t stream) {
    constexpr int HQ = 1, HP = 1;
    const int64_t np = (a.J + HP * 128 - 1) / (HP * 128);
    int64_t nq;
    if (MODE == kDw)
        nq = (a.I + HQ * 128 - 1) / (HQ * 128) * a.L;
    else if (MODE == kI8)
        nq = (a.T + HQ * 128 - 1) / (HQ * 128);
    else
        nq = a.T / (HQ * 128) + a.L + 2;
    const int64_t wgs = (nq * np + 7) / 8 * 8;
    if (wgs >= ((int64_t)1 << 31)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((prod_tile_kernel<MODE, HQ, HP, DMA>), dim3((uint32_t)wgs), dim3(kNT), 0, stream, a);
    return hipGetLastError();
}

template <int MODE>
hipError_t launch_prod(const ProdArgs& a, hipStream_t stream) {
    const int e = MODE == kI8 ? 1 : 2;
    bool whole;
    if (MODE == kDw)
        whole = chunked(a.q, a.qs, a.I * e) && chunked(a.p, a.ps, a.J * e);
    else if (MODE == kDx)
        whole = chunked(a.q, a.qs, a.red * e) && chunked(a.p, a.ps, a.J * e);
    else
        whole = chunked(a.q, a.qs, a.red * e) && chunked(a.p, a.ps, 0);
    return whole ? launch_tiles<MODE, true>(a, stream) : launch_tiles<MODE, false>(a, stream);
}

}  // namespace

hipError_t launch_i8_quantize(const void* x, int32_t dtype, int64_t n, int32_t d, int64_t xs, int8_t* codes,
                              float* scale, hipStream_t stream) {
    const uint32_t wgs = (uint32_t)(n < 65536 ? n : 65536);
    if (dtype == AH_F32)
        hipLaunchKernelGGL(i8_quantize_kernel<float>, dim3(wgs), dim3(256), 0, stream, static_cast<const float*>(x), n,
                           d, xs, codes, scale);
    else
        hipLaunchKernelGGL(i8_quantize_kernel<uint16_t>, dim3(wgs), dim3(256), 0, stream,
                           static_cast<const uint16_t*>(x), n, d, xs, codes, scale);
    return hipGetLastError();
}

hipError_t launch_i8_matmul(const int8_t* x8, const float* xs, int64_t m, const int8_t* w8, const float* ws, int64_t n,
                            int32_t k, const float* bias, void* out, int32_t out_dtype, hipStream_t stream) {
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
    return launch_prod<kI8>(a, stream);
}

// Workspace: the tokens' codes (rows of k bytes, the block rounded up to 16) and their steps.
static size_t code_bytes(int64_t m, int32_t k) { return ((size_t)m * k + 15) / 16 * 16; }
size_t i8_linear_workspace_bytes(int64_t m, int32_t k) { return code_bytes(m, k) + (size_t)m * sizeof(float); }

hipError_t launch_i8_linear(const void* x, int32_t dtype, int64_t m, int32_t k, int64_t xs, const int8_t* w8,
                            const float* ws, int64_t n, const float* bias, void* out, int32_t out_dtype, void* work,
                            hipStream_t stream) {
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
    a.fan = g.fan;
    a.J = g.n;
    a.red = g.k;
    a.out = out;
    a.out_f32 = out_dtype == AH_F32;
    return launch_prod<kFwd>(a, stream);
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
    a.fan = g.fan;
    a.J = g.k;
    a.red = g.n;
    a.out = g.fan > 1 ? ws : out;
    a.out_f32 = g.fan > 1 || out_dtype == AH_F32;
    hipError_t e = launch_prod<kDx>(a, stream);
    if (e != hipSuccess || g.fan == 1) return e;
    const int64_t rows = g.slots / g.fan, wgs = (rows * g.k + 255) / 256;
    hipLaunchKernelGGL(fan_sum_kernel, dim3((uint32_t)(wgs < 8192 ? wgs : 8192)), dim3(256), 0, stream,
                       static_cast<const float*>(ws), rows, g.fan, (int64_t)g.k, out, out_dtype == AH_F32);
    return hipGetLastError();
}

hipError_t launch_grouped_dw(const GroupedProblem& g, void* out, int32_t out_dtype, hipStream_t stream) {
    ProdArgs a{};
    a.q = static_cast<const char*>(g.dy);
    a.qs = g.dy_stride * 2;
    a.p = static_cast<const char*>(g.x);
    a.ps = g.x_stride * 2;
    a.off = g.offsets;
    a.order = g.order;
    a.T = g.slots;
    a.I = g.n;
    a.L = g.L;
    a.fan = g.fan;
    a.J = g.k;
    a.out = out;
    a.out_f32 = out_dtype == AH_F32;
    return launch_prod<kDw>(a, stream);
}

}  // namespace ah
