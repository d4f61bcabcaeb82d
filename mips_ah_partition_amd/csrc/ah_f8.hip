// Products in 8-bit floating point (e4m3 or e5m2) with a power-of-two scale for each block of 128 along the sum: the
// codes, the product of few rows, and the tiled one of ah_tiles.hpp.
#include "ah_tiles.hpp"

namespace ah {
namespace {

constexpr int kBlk = 128;

// Scale byte of a block whose largest |x| is m: e + 127 for the smallest e (from -127 on) with m 2^-e at most the
// type's largest value, 1.75 2^8 or 1.75 2^15.  With m = f 2^t, f in [1, 2), that is t - 8 (15), and one more where f > 1.75.
__device__ __forceinline__ int scale_byte(float m, int type) {
    if (!(m > 0.0f)) return 127;
    int t;
    const float f = frexpf(m, &t);  // in [0.5, 1)
    const int e = t + (f > 0.875f ? 1 : 0) - (type == AH_E4M3 ? 9 : 16) + 127;
    return e < 0 ? 0 : e;
}
// 2^-e of a scale byte (at most 247: a float32 below 2^128).
__device__ __forceinline__ float inverse_of(int s) { return __uint_as_float((uint32_t)(254 - s) << 23); }

// Four values to codes, rounded to nearest even.
template <int TYPE>
__device__ __forceinline__ int codes4(const float* v) {
    int r = 0;
    if constexpr (TYPE == AH_E4M3) {
        r = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], r, false);
        r = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], r, true);
    } else {
        r = __builtin_amdgcn_cvt_pk_bf8_f32(v[0], v[1], r, false);
        r = __builtin_amdgcn_cvt_pk_bf8_f32(v[2], v[3], r, true);
    }
    return r;
}
// A block's scale byte and the factor of its values; m +inf: a NaN or an infinity in it, codes are NaN.
struct BlockScale {
    int byte;
    float inv;
    bool bad;
};
__device__ __forceinline__ BlockScale block_scale(float m, int type) {
    const bool bad = !(m < INFINITY);
    const int s = bad ? 127 : scale_byte(m, type);
    return BlockScale{s, inverse_of(s), bad};
}
template <int TYPE>
__device__ __forceinline__ int codes4(const float* v, const BlockScale& s) {
    float t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = v[e] * s.inv;
    return s.bad ? 0x7F7F7F7F : codes4<TYPE>(t);
}

// Eight elements of a row from element c on, as float32; zeros past its d elements.
template <typename T, bool WHOLE>
__device__ __forceinline__ void load8(const T* row, int64_t c, int64_t d, float* v) {
    constexpr int N = sizeof(T) / 2;  // chunks of 16 bytes
    T e[8];
#pragma unroll
    for (int h = 0; h < N; ++h) {
        const char* p = reinterpret_cast<const char*>(row + c) + h * 16;
        v4i x = {0, 0, 0, 0};
        if constexpr (WHOLE) {
            if (c + h * 4 < d) x = *reinterpret_cast<const v4i*>(p);
        } else {
            x = load_chunk<sizeof(T)>(p, (d - c) * (int64_t)sizeof(T) - h * 16, c * (int64_t)sizeof(T) + h * 16);
        }
        __builtin_memcpy(reinterpret_cast<char*>(e) + h * 16, &x, 16);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
}
__device__ __forceinline__ float largest(const float* v, int n) {  // +inf where one is NaN or infinite
    float m = 0.0f;
    bool bad = false;
    for (int i = 0; i < n; ++i) {
        const float f = fabsf(v[i]);
        bad |= !(f < INFINITY);
        m = fmaxf(m, f);
    }
    return bad ? INFINITY : m;
}

// Rows to codes.  HBM-bound (2 or 4 bytes in, 1 out; bfloat16 8192 x 4096: 24 us, 4.2 TB/s).  16 lanes have a block of
// 128, 8 elements each (one or two loads of 16 bytes and a store of 8), a wave four blocks of a row: no barrier, no LDS.
template <typename T, int TYPE, bool WHOLE>
__global__ __launch_bounds__(256) void f8_rows_kernel(const T* x, int64_t n, int64_t d, int64_t xs, uint8_t* codes,
                                                      uint8_t* scale) {
    const int lane = threadIdx.x & 63;
    const int64_t kb = (d + kBlk - 1) / kBlk, pitch = (n + 15) / 16 * 16, per = (kb + 3) / 4, items = n * per;
    for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < items; i += (int64_t)gridDim.x * 4) {
        const int64_t r = i / per, b = (i - r * per) * 4 + (lane >> 4), c = b * kBlk + (lane & 15) * 8;
        float v[8];
        load8<T, WHOLE>(x + r * xs, c, d, v);
        float m = largest(v, 8);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
        const BlockScale s = block_scale(m, TYPE);
        if (b < kb) {
            const int w[2] = {codes4<TYPE>(v, s), codes4<TYPE>(v + 4, s)};
            const int64_t left = d - c;  // zeros past the row, also in a bad block
            uint64_t u = (uint32_t)w[0] | (uint64_t)(uint32_t)w[1] << 32;
            if (left < 8) u = left <= 0 ? 0 : u & ((1ull << (8 * left)) - 1);
            *reinterpret_cast<uint64_t*>(codes + r * kb * kBlk + c) = u;
            if ((lane & 15) == 0) scale[b * pitch + r] = (uint8_t)s.byte;
        }
    }
}

// Columns to codes (the transposed matrix), and rows too where wanted, from one reading: a workgroup has 128 x 128
// elements, its rows' blocks in registers, its columns' through LDS, 32 elements of a column a thread.  Bfloat16 8192 x
// 4096 to both: 33-36 us (134 MB, 4.0 TB/s; two passes would read 67 MB more), 8192 x 1536 to columns 11.6; 256 threads, 64
// elements of a column each: 36, and 500 x 77 9.1 instead of 6.1.  Bound by the memory and the two barriers a tile.
constexpr int kColThreads = 512, kParts = kColThreads / kBlk, kPart = kBlk / kParts;
template <typename T, int TYPE, bool WHOLE, bool ROWS>
__global__ __launch_bounds__(kColThreads) void f8_columns_kernel(const T* x, int64_t n, int64_t d, int64_t xs, uint8_t* codes,
                                                         uint8_t* scale, uint8_t* codes_t, uint8_t* scale_t) {
    __shared__ __align__(16) T tile[kBlk][kBlk + 8];
    __shared__ float most[kParts][kBlk];
    const int tid = threadIdx.x;
    const int64_t kb = (d + kBlk - 1) / kBlk, nb = (n + kBlk - 1) / kBlk;
    const int64_t pitch = (n + 15) / 16 * 16, pitch_t = (d + 15) / 16 * 16;
    for (int64_t i = blockIdx.x; i < kb * nb; i += gridDim.x) {
        const int64_t r0 = i / kb * kBlk, b = i % kb, c0 = b * kBlk, c = c0 + (tid & 15) * 8;
#pragma unroll
        for (int k = 0; k < kBlk * 16 / kColThreads; ++k) {
            const int rr = k * (kColThreads / 16) + (tid >> 4);
            const int64_t r = r0 + rr;
            float v[8] = {};
            if (r < n) load8<T, WHOLE>(x + r * xs, c, d, v);
            T raw[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (sizeof(T) == 4)
                    raw[e] = v[e];
                else
                    raw[e] = (T)(__float_as_uint(v[e]) >> 16);
            }
            __builtin_memcpy(&tile[rr][(tid & 15) * 8], raw, sizeof(raw));
            if constexpr (ROWS) {
                float m = largest(v, 8);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
                const BlockScale s = block_scale(m, TYPE);
                if (r < n) {
                    const int w[2] = {codes4<TYPE>(v, s), codes4<TYPE>(v + 4, s)};
                    uint64_t u = (uint32_t)w[0] | (uint64_t)(uint32_t)w[1] << 32;
                    const int64_t left = d - c;
                    if (left < 8) u = left <= 0 ? 0 : u & ((1ull << (8 * left)) - 1);
                    *reinterpret_cast<uint64_t*>(codes + r * kb * kBlk + c) = u;
                    if ((tid & 15) == 0) scale[b * pitch + r] = (uint8_t)s.byte;
                }
            }
        }
        __syncthreads();
        const int cc = tid & 127, h = tid >> 7;
        float v[kPart];
#pragma unroll
        for (int k = 0; k < kPart; ++k) v[k] = to_f32(tile[h * kPart + k][cc]);
        most[h][cc] = largest(v, kPart);
        __syncthreads();
        float m = most[0][cc];
#pragma unroll
        for (int k = 1; k < kParts; ++k) m = fmaxf(m, most[k][cc]);
        const BlockScale s = block_scale(m, TYPE);
        if (c0 + cc < d) {
            uint8_t* const o = codes_t + (c0 + cc) * nb * kBlk + r0 + h * kPart;
#pragma unroll
            for (int k = 0; k < kPart; k += 16) {
                v4i w;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    w[q] = codes4<TYPE>(v + k + q * 4, s);
                    if (s.bad) {  // zeros past the last row
                        const int64_t left = n - (r0 + h * kPart + k + q * 4);
                        if (left < 4) w[q] = left <= 0 ? 0 : w[q] & ((1 << (8 * (int)left)) - 1);
                    }
                }
                *reinterpret_cast<v4i*>(o + k) = w;
            }
            if (h == 0) scale_t[r0 / kBlk * pitch_t + c0 + cc] = (uint8_t)s.byte;
        }
        __syncthreads();
    }
}

// Few rows or few columns (few_fragments): few rows are one pass over the weights.  A workgroup has 16 columns and 16 FR
// rows; its eight waves share out the steps of 128, load both operands from memory into the matrix instruction's layout
// (lane 16 g + i: bytes 16 g .. and 64 + 16 g .. of row i) and add up through LDS in a fixed order.  XB = 2 or 4: the rows
// are of that many bytes an element, and every workgroup turns them to codes for itself (a block's largest value lies in
// four lanes of the wave that needs it, so nothing waits): one launch instead of two.  One row, 1536 -> 4096: 6.0-6.5 us
// on the GPU, a launch and the chain of loads, codes, sum and exchange (6.4 MB of weights are 1.2); a call 10.0, 12.1 with a
// launch to quantise.  Up to 16 rows (kFewRows, with its figures): of 37 x 1001 it took 12.4 us on the GPU, quantising and
// product in turn 3.2 + 5.4.  whole: their chunks of 16 bytes are aligned and 16 elements inside the row or outside together.
template <int XT, int WT, int FR, int XB>
__global__ __launch_bounds__(kRowWaves * 64) void f8_few_kernel(ProdArgs a, int64_t k, bool whole) {
    constexpr int U = FR == 4 ? 2 : 4, MODE = kF8 + XT + 2 * WT;
    static_assert(XB == 0 || FR == 1, "");
    __shared__ v4f part[kRowWaves][FR][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, li = lane & 15;
    const int32_t steps = (int32_t)(a.red / kBlk), s0 = (int32_t)((int64_t)steps * wave / kRowWaves),
                  s1 = (int32_t)((int64_t)steps * (wave + 1) / kRowWaves);
    const int64_t j0 = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * 16, j = j0 + g * 4, p0 = (int64_t)blockIdx.y * 16 * FR;
    if (j0 >= a.J) return;
    const int64_t col = j0 + li < a.J ? j0 + li : a.J - 1;
    const char* const prow = a.p + col * a.ps + g * 16;
    const char* const psc = a.psc + col;
    const char* qrow[FR];
    const char* qsc[FR];
#pragma unroll
    for (int f = 0; f < FR; ++f) {
        const int64_t r = p0 + f * 16 + li < a.T ? p0 + f * 16 + li : a.T - 1;  // rows past the last repeat it
        qrow[f] = a.q + r * a.qs + g * 16 * (XB ? XB : 1);
        if constexpr (XB == 0) qsc[f] = a.qsc + r;
    }
    float bias[4] = {};
    if (wave < FR && a.bias) {
#pragma unroll
        for (int e = 0; e < 4; ++e) bias[e] = a.bias[j + e < a.J ? j + e : a.J - 1];
    }
    v4f acc[FR];
#pragma unroll
    for (int f = 0; f < FR; ++f) acc[f] = v4f{0, 0, 0, 0};
    for (int32_t s = s0; s < s1; s += U) {
        v4i pv[U][2], qv[U][FR][2], xv[XB ? U : 1][FR][XB ? 2 * XB : 1];
        int sp[U], sq[U][FR];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s + u < s1) {
                const int64_t o = (int64_t)(s + u) * kBlk;
                sp[u] = *reinterpret_cast<const uint8_t*>(psc + (s + u) * a.ppitch);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (XB == 0) {
#pragma unroll
                        for (int f = 0; f < FR; ++f) qv[u][f][h] = *reinterpret_cast<const v4i*>(qrow[f] + o + h * 64);
                    } else {  // 16 elements
                        const int64_t left = k - (o + h * 64 + g * 16);
#pragma unroll
                        for (int f = 0; f < FR; ++f)
#pragma unroll
                            for (int c = 0; c < XB; ++c) {
                                const char* const p = qrow[f] + (o + h * 64) * XB + c * 16;
                                if (whole)
                                    xv[u][f][h * XB + c] = left > 0 ? *reinterpret_cast<const v4i*>(p) : v4i{0, 0, 0, 0};
                                else
                                    xv[u][f][h * XB + c] = load_chunk<XB>(p, left * XB - c * 16, (k - left) * XB + c * 16);
                            }
                    }
                    pv[u][h] = *reinterpret_cast<const v4i*>(prow + o + h * 64);
                }
                if constexpr (XB == 0) {
#pragma unroll
                    for (int f = 0; f < FR; ++f) sq[u][f] = *reinterpret_cast<const uint8_t*>(qsc[f] + (s + u) * a.qpitch);
                }
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s + u < s1) {
                if constexpr (XB > 0) {
                    typedef typename std::conditional<XB == 2, uint16_t, float>::type T;
#pragma unroll
                    for (int f = 0; f < FR; ++f) {
                        T e[32];
                        __builtin_memcpy(e, xv[u][f], sizeof(e));
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = to_f32(e[i]);
                        float m = largest(v, 32);
                        m = fmaxf(m, __shfl_xor(m, 16, 64));
                        m = fmaxf(m, __shfl_xor(m, 32, 64));
                        const BlockScale b = block_scale(m, XT);
                        sq[u][f] = b.byte;
#pragma unroll
                        for (int i = 0; i < 8; ++i) qv[u][f][i >> 2][i & 3] = codes4<XT>(v + i * 4, b);
                    }
                }
#pragma unroll
                for (int f = 0; f < FR; ++f)
                    acc[f] = mma8<MODE>(halves(pv[u][0], pv[u][1]), halves(qv[u][f][0], qv[u][f][1]), acc[f], sp[u], sq[u][f]);
            }
    }
#pragma unroll
    for (int f = 0; f < FR; ++f) part[wave][f][lane] = acc[f];
    __syncthreads();
#pragma unroll
    for (int f = 0; f < FR; ++f) {
        const int64_t row = p0 + f * 16 + li, left = a.J - j;
        if (wave != f || row >= a.T || left <= 0) continue;
        v4f t = part[0][f][lane];
#pragma unroll
        for (int w = 1; w < kRowWaves; ++w) t += part[w][f][lane];
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = t[e] + bias[e];
        const int32_t some = left < 4 ? (int32_t)left : 4;
        if (a.out_f32) {
            char* const o = static_cast<char*>(a.out) + (row * a.J + j) * 4;
            v4i w;
            __builtin_memcpy(&w, y, 16);
            if (some == 4)
                __builtin_memcpy(o, &w, 16);
            else
                store_left<4>(o, w, some);
        } else {
            put_bf16(static_cast<char*>(a.out) + (row * a.J + j) * 2, y, some);
        }
    }
}

ProdArgs f8_args(const F8Problem& g, const float* bias, void* out, int32_t out_dtype) {
    const int64_t kp = (g.k + kBlk - 1) / kBlk * kBlk;
    ProdArgs a{};
    a.q = reinterpret_cast<const char*>(g.x8);
    a.p = reinterpret_cast<const char*>(g.w8);
    a.qs = a.ps = kp;
    a.T = a.I = g.m;
    a.J = g.n;
    a.red = kp;
    a.out = out;
    a.out_f32 = out_dtype == AH_F32;
    a.bias = bias;
    a.qsc = reinterpret_cast<const char*>(g.xs);
    a.psc = reinterpret_cast<const char*>(g.ws);
    a.qpitch = (g.m + 15) / 16 * 16;
    a.ppitch = (g.n + 15) / 16 * 16;
    return a;
}

template <int XT, int WT, int FR, int XB>
hipError_t launch_few(const ProdArgs& a, int64_t k, bool whole, hipStream_t stream) {
    const int64_t strips = (a.J + 15) / 16, most = kMaxGridItems / (kRowWaves * 64);  // of one launch dimension
    const int64_t z = (strips + most - 1) / most;
    const dim3 grid((uint32_t)((strips + z - 1) / z), (uint32_t)((a.T + 16 * FR - 1) / (16 * FR)), (uint32_t)z);
    hipLaunchKernelGGL((f8_few_kernel<XT, WT, FR, XB>), grid, dim3(kRowWaves * 64), 0, stream, a, k, whole);
    return hipGetLastError();
}

// Row fragments of f8_few_kernel, or 0 for tiles, which take `tiles` us (f8_shape): its time is a chain of loads and matrix
// instructions for every eight steps and the start of its workgroups, or what they read, from L2 mostly, each 16 columns and
// 16 FR rows.  Few columns and long sums are its own, however many the rows; many columns of more than 16 rows are the
// tiles'.  Measured, us, FR = 1, 2, 4 and the tiles:
//   100 x 8192 x 100       9.6   13.5   20.7   28.0          64 x 4096 x 4096      17.7   15.2   12.8   15.7
//   300 x 4096 x 300       9.8    8.3   12.0   16.2          64 x 4096 x 16384     61.2   53.6   45.2   16.7
//   500 x 200 x 77         2.9    3.1    3.5    4.4          333 x 4096 x 1001     24.7   21.7   23.6   16.0
//   256 x 768 x 384        3.9    3.8    4.6    5.9          1024 x 768 x 384       7.9    7.6    7.8    5.9
int few_fragments(const ProdArgs& a, double tiles) {
    if (a.T <= 16) return 1;  // as ah_f8_linear's product that quantises, whose sums are to be the same
    const struct {
        int fr;
        double chain, starts, rate;  // us for every eight steps, workgroups a us beyond one a CU, MB a us
    } few[] = {{1, 0.9, 420, 7.0}, {2, 1.4, 200, 5.5}, {4, 2.3, 60, 7.0}};
    int best = 0;
    for (const auto& f : few) {
        const int64_t rows = (a.T + 16 * f.fr - 1) / (16 * f.fr), wgs = rows * ((a.J + 15) / 16),
                      steps = (a.red + 127) / 128;
        const double start = (double)((steps + kRowWaves - 1) / kRowWaves) * f.chain +
                             (wgs > kCUs ? (double)(wgs - kCUs) / f.starts : 0.0),
                     read = (double)wgs * 16 * (1 + f.fr) * (double)a.red * 1e-6 / f.rate,
                     time = 2.0 + (start > read ? start : read);
        if (rows <= 65535 && time < tiles) {  // (a launch's second dimension)
            best = f.fr;
            tiles = time;
        }
    }
    return best;
}

template <int XT, int WT>
hipError_t launch_types(const ProdArgs& a, int64_t k, hipStream_t stream) {
    constexpr int MODE = kF8 + XT + 2 * WT;
    double tiles;
    f8_shape<MODE>(a, &tiles);
    switch (few_fragments(a, tiles + 2.0)) {  // (a launch)
        case 1: return launch_few<XT, WT, 1, 0>(a, k, true, stream);
        case 2: return launch_few<XT, WT, 2, 0>(a, k, true, stream);
        case 4: return launch_few<XT, WT, 4, 0>(a, k, true, stream);
        default: return launch_prod<MODE>(a, 1, stream);
    }
}

hipError_t launch_f8(const F8Problem& g, const ProdArgs& a, hipStream_t stream) {
    if (g.x_type == AH_E4M3)
        return g.w_type == AH_E4M3 ? launch_types<AH_E4M3, AH_E4M3>(a, g.k, stream)
                                   : launch_types<AH_E4M3, AH_E5M2>(a, g.k, stream);
    return g.w_type == AH_E4M3 ? launch_types<AH_E5M2, AH_E4M3>(a, g.k, stream)
                               : launch_types<AH_E5M2, AH_E5M2>(a, g.k, stream);
}

template <typename T, int TYPE>
hipError_t launch_quantize(const T* x, int64_t n, int64_t d, int64_t xs, uint8_t* codes, uint8_t* scale,
                           uint8_t* codes_t, uint8_t* scale_t, hipStream_t stream) {
    const bool whole = chunked(x, xs * (int64_t)sizeof(T), 0) && d % 8 == 0;
    const int64_t kb = (d + kBlk - 1) / kBlk;
    if (!codes_t) {
        const int64_t wgs = (n * ((kb + 3) / 4) + 3) / 4;
        const dim3 grid((uint32_t)(wgs < (1 << 20) ? wgs : 1 << 20));
        auto kernel = whole ? f8_rows_kernel<T, TYPE, true> : f8_rows_kernel<T, TYPE, false>;
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, x, n, d, xs, codes, scale);
    } else {
        const int64_t wgs = (n + kBlk - 1) / kBlk * kb;
        const dim3 grid((uint32_t)(wgs < (1 << 20) ? wgs : 1 << 20));
        auto kernel = codes ? (whole ? f8_columns_kernel<T, TYPE, true, true> : f8_columns_kernel<T, TYPE, false, true>)
                            : (whole ? f8_columns_kernel<T, TYPE, true, false> : f8_columns_kernel<T, TYPE, false, false>);
        hipLaunchKernelGGL(kernel, grid, dim3(kColThreads), 0, stream, x, n, d, xs, codes, scale, codes_t, scale_t);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_quantize(const void* x, int32_t dtype, int64_t n, int64_t d, int64_t xs, int32_t type,
                              uint8_t* codes, uint8_t* scale, uint8_t* codes_t, uint8_t* scale_t, hipStream_t stream) {
    auto go = [&](auto* rows) {
        return type == AH_E4M3 ? launch_quantize<std::remove_const_t<std::remove_pointer_t<decltype(rows)>>, AH_E4M3>(
                                     rows, n, d, xs, codes, scale, codes_t, scale_t, stream)
                               : launch_quantize<std::remove_const_t<std::remove_pointer_t<decltype(rows)>>, AH_E5M2>(
                                     rows, n, d, xs, codes, scale, codes_t, scale_t, stream);
    };
    return dtype == AH_F32 ? go(static_cast<const float*>(x)) : go(static_cast<const uint16_t*>(x));
}

hipError_t launch_f8_matmul(const F8Problem& g, const float* bias, void* out, int32_t out_dtype, hipStream_t stream) {
    return launch_f8(g, f8_args(g, bias, out, out_dtype), stream);
}

// Workspace: the rows' codes, then their scale bytes; none for rows that the product turns to codes itself.
// Measured, us, codes in the product | in a launch of their own (2, 8 and 16 rows; on the GPU, then a call):
//   1536 -> 4096    5.7  6.0  6.4 | 5.7  6.0  6.4      9.5  9.5  9.5 | 18.7 18.8 18.8
//   4096 -> 16384   38.6 40.5 43.6 | 17.2 18.5 20.7    37.9 40.3 43.1 | 18.7 18.6 20.5
// One fragment of rows is what every workgroup can keep; wide layers, where each of many workgroups makes the same codes again,
// would be faster by two launches, which the rule does not tell apart.
constexpr int64_t kFewRows = 16;
static size_t f8_code_bytes(int64_t m, int64_t k) { return (size_t)m * ((k + kBlk - 1) / kBlk * kBlk); }
size_t f8_linear_workspace_bytes(int64_t m, int64_t k) {
    return m <= kFewRows ? 0 : f8_code_bytes(m, k) + (size_t)((k + kBlk - 1) / kBlk) * ((m + 15) / 16 * 16);
}

hipError_t launch_f8_linear(const void* x, int32_t dtype, int64_t xs, const F8Problem& p, const float* bias, void* out,
                            int32_t out_dtype, void* work, hipStream_t stream) {
    const int64_t bytes = dtype == AH_F32 ? 4 : 2;
    if (p.m <= kFewRows) {
        const bool whole = chunked(x, xs * bytes, 0) && p.k % 16 == 0;
        ProdArgs a = f8_args(p, bias, out, out_dtype);
        a.q = static_cast<const char*>(x);
        a.qs = xs * bytes;
        auto go = [&](auto xt, auto wt) {
            return dtype == AH_F32 ? launch_few<decltype(xt)::value, decltype(wt)::value, 1, 4>(a, p.k, whole, stream)
                                   : launch_few<decltype(xt)::value, decltype(wt)::value, 1, 2>(a, p.k, whole, stream);
        };
        const std::integral_constant<int, AH_E4M3> e4;
        const std::integral_constant<int, AH_E5M2> e5;
        if (p.x_type == AH_E4M3) return p.w_type == AH_E4M3 ? go(e4, e4) : go(e4, e5);
        return p.w_type == AH_E4M3 ? go(e5, e4) : go(e5, e5);
    }
    F8Problem g = p;
    uint8_t* codes = static_cast<uint8_t*>(work);
    uint8_t* scale = codes + f8_code_bytes(p.m, p.k);
    g.x8 = codes;
    g.xs = scale;
    const hipError_t e = launch_f8_quantize(x, dtype, p.m, p.k, xs, p.x_type, codes, scale, nullptr, nullptr, stream);
    if (e != hipSuccess) return e;
    return launch_f8_matmul(g, bias, out, out_dtype, stream);
}

}  // namespace ah
