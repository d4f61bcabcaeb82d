// Dropout with a mask that is computed and never stored, and the addition of a residual.
#include "ah_device.hpp"
#include "ah_kernels.hpp"
#include "ah_random.hpp"
#include "../../include/ah.h"

namespace ah {
namespace {

template <typename T>
__device__ __forceinline__ float wide(T v) {
    if constexpr (sizeof(T) == 4)
        return v;
    else
        return __uint_as_float((uint32_t)v << 16);
}
template <typename T>
__global__ __launch_bounds__(256) void dropout_kernel(const T* x, int64_t rows, int64_t n, int64_t xs, Dropout d,
                                                      const T* res, int64_t rs, T* out, int64_t os) {
    const uint64_t step = d.t ? step_of_call(d) : 0;
    const int64_t per = (n + 7) / 8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * per; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per, c = i % per;
        const Philox u = philox(d, step, (uint32_t)r, (uint32_t)c);
        for (int j = 0; j < 8 && c * 8 + j < n; ++j) {
            float v = wide(x[r * xs + c * 8 + j]);
            v = u.at(j) >= d.t ? v * d.factor : 0.0f;
            if (res) v += wide(res[r * rs + c * 8 + j]);
            if constexpr (sizeof(T) == 4)
                out[r * os + c * 8 + j] = v;
            else
                out[r * os + c * 8 + j] = __builtin_bit_cast(uint16_t, (__bf16)v);
        }
    }
}

}  // namespace

hipError_t launch_dropout(const void* x, int32_t dtype, int64_t rows, int64_t n, int64_t xs, const Dropout& d,
                          const void* res, int64_t rs, void* out, int64_t os, hipStream_t stream) {
    const int64_t items = rows * ((n + 7) / 8), wgs = (items + 255) / 256;
    const dim3 grid((uint32_t)(wgs < 65536 ? wgs : 65536));
    if (dtype == AH_F32)
        hipLaunchKernelGGL(dropout_kernel<float>, grid, dim3(256), 0, stream, static_cast<const float*>(x), rows, n, xs,
                           d, static_cast<const float*>(res), rs, static_cast<float*>(out), os);
    else
        hipLaunchKernelGGL(dropout_kernel<uint16_t>, grid, dim3(256), 0, stream, static_cast<const uint16_t*>(x), rows,
                           n, xs, d, static_cast<const uint16_t*>(res), rs, static_cast<uint16_t*>(out), os);
    return hipGetLastError();
}

}  // namespace ah
