// Products in 8-bit floating point (e4m3 or e5m2) with a power-of-two scale for each block of 128 along the sum.
#include "ah_device.hpp"
#include "ah_kernels.hpp"
#include "ah_simple.hpp"
#include "../../include/ah.h"

namespace ah {
namespace {

constexpr int kBlk = 128;
__device__ __forceinline__ float f32_in(const void* x, int f32, int64_t i) {
    return f32 ? static_cast<const float*>(x)[i] : __uint_as_float((uint32_t)static_cast<const uint16_t*>(x)[i] << 16);
}
// Scale byte of a block whose largest |x| is m (+inf: a NaN or an infinity among them).
__device__ __forceinline__ int scale_byte(float m, int type) {
    if (!(m > 0.0f)) return 127;
    int e;
    const float f = frexpf(m, &e);  // m = f 2^e, f in [0.5, 1); the types' largest values: 0.875 2^9 and 0.875 2^16
    e += (f > 0.875f ? 1 : 0) - (type == AH_E4M3 ? 9 : 16) + 127;
    return e < 0 ? 0 : e;
}
__device__ __forceinline__ uint8_t code_of(float v, int type) {
    return (uint8_t)(type == AH_E4M3 ? __builtin_amdgcn_cvt_pk_fp8_f32(v, 0.0f, 0, false)
                                     : __builtin_amdgcn_cvt_pk_bf8_f32(v, 0.0f, 0, false));
}
// One thread a block of 128 elements, `es` apart.
__global__ void f8_quantize_kernel(const void* x, int f32, int64_t rows, int64_t len, int64_t rs, int64_t es, int type,
                                   uint8_t* codes, uint8_t* scale) {
    const int64_t kb = (len + kBlk - 1) / kBlk, pitch = (rows + 15) / 16 * 16;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pitch * kb; i += (int64_t)gridDim.x * 256) {
        const int64_t b = i / pitch, r = i % pitch, t1 = len - b * kBlk < kBlk ? len - b * kBlk : kBlk;
        if (r >= rows) {
            scale[i] = 127;
            continue;
        }
        float m = 0.0f;
        for (int64_t t = 0; t < t1; ++t) {
            const float v = fabsf(f32_in(x, f32, r * rs + (b * kBlk + t) * es));
            m = v < INFINITY ? fmaxf(m, v) : INFINITY;
            if (!(v < INFINITY)) break;
        }
        uint8_t* c = codes + (r * kb + b) * kBlk;
        const bool bad = !(m < INFINITY);
        const int s = bad ? 127 : scale_byte(m, type);
        scale[i] = (uint8_t)s;
        for (int64_t t = 0; t < kBlk; ++t)
            c[t] = t >= t1 ? 0 : bad ? 0x7F : code_of(ldexpf(f32_in(x, f32, r * rs + (b * kBlk + t) * es), 127 - s), type);
    }
}
__device__ __forceinline__ float value_of(uint8_t c, int type) {
    return type == AH_E4M3 ? __builtin_amdgcn_cvt_f32_fp8((int)c, 0) : __builtin_amdgcn_cvt_f32_bf8((int)c, 0);
}
__global__ __launch_bounds__(256) void f8_product_kernel(F8Problem g, const float* bias, void* out, int out_f32) {
    const int64_t kb = (g.k + kBlk - 1) / kBlk, pm = (g.m + 15) / 16 * 16, pn = (g.n + 15) / 16 * 16;
    const int64_t j0 = (int64_t)blockIdx.x * 64;
    for (int64_t i0 = (int64_t)blockIdx.y * 64; i0 < g.m; i0 += (int64_t)gridDim.y * 64)
        simple_tile<1>(
            kb * kBlk,
            [&](int r, int64_t t) {
                const int64_t i = i0 + r;
                return i < g.m ? ldexpf(value_of(g.x8[i * kb * kBlk + t], g.x_type), g.xs[t / kBlk * pm + i] - 127) : 0.0f;
            },
            [&](int, int c, int64_t t) {
                const int64_t j = j0 + c;
                return j < g.n ? ldexpf(value_of(g.w8[j * kb * kBlk + t], g.w_type), g.ws[t / kBlk * pn + j] - 127) : 0.0f;
            },
            [&](int r, int c, const float* v) {
                const int64_t i = i0 + r, j = j0 + c;
                if (i >= g.m || j >= g.n) return;
                const float y = v[0] + (bias ? bias[j] : 0.0f);
                if (out_f32)
                    static_cast<float*>(out)[i * g.n + j] = y;
                else
                    static_cast<uint16_t*>(out)[i * g.n + j] = __builtin_bit_cast(uint16_t, (__bf16)y);
            });
}

}  // namespace

hipError_t launch_f8_quantize(const void* x, int32_t dtype, int64_t n, int64_t d, int64_t xs, int32_t type,
                              uint8_t* codes, uint8_t* scale, uint8_t* codes_t, uint8_t* scale_t, hipStream_t stream) {
    if (codes)
        hipLaunchKernelGGL(f8_quantize_kernel, dim3(4096), dim3(256), 0, stream, x, dtype == AH_F32, n, d, xs,
                           (int64_t)1, type, codes, scale);
    if (codes_t)
        hipLaunchKernelGGL(f8_quantize_kernel, dim3(4096), dim3(256), 0, stream, x, dtype == AH_F32, d, n, (int64_t)1,
                           xs, type, codes_t, scale_t);
    return hipGetLastError();
}

hipError_t launch_f8_matmul(const F8Problem& g, const float* bias, void* out, int32_t out_dtype, hipStream_t stream) {
    const int64_t rows = (g.m + 63) / 64;
    hipLaunchKernelGGL(f8_product_kernel, dim3((uint32_t)((g.n + 63) / 64), (uint32_t)(rows < 1024 ? rows : 1024)),
                       dim3(256), 0, stream, g, bias, out, out_dtype == AH_F32);
    return hipGetLastError();
}

static size_t f8_code_bytes(int64_t m, int64_t k) { return (size_t)m * ((k + kBlk - 1) / kBlk * kBlk); }
size_t f8_linear_workspace_bytes(int64_t m, int64_t k) {
    return f8_code_bytes(m, k) + (size_t)((k + kBlk - 1) / kBlk) * ((m + 15) / 16 * 16);
}

hipError_t launch_f8_linear(const void* x, int32_t dtype, int64_t xs, const F8Problem& p, const float* bias, void* out,
                            int32_t out_dtype, void* work, hipStream_t stream) {
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
