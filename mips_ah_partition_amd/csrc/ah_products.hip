// Int8 rows with a scale for each token and channel, and bfloat16 rows grouped by leaf (every leaf of a
// partition has its own weight matrix) with their gradients: the products of ah_tiles.hpp.
#include "ah_tiles.hpp"

namespace ah {
namespace {

// Rows to codes (step_of, chunk_codes).  HBM-bound (2 or 4 bytes in, 1 out; bfloat16 8192 x 4096: 23 us, 4.3 TB/s;
// float32 40 us, 4.2): one wave per row, no barrier; the row is read once and kept in registers up to 8 chunks of 16
// bytes a lane.  WHOLE: the rows are whole aligned chunks; else chunks at any alignment, the last one short.
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
