// Dropout with a mask that is computed and never stored, and the addition of a residual.
#include <type_traits>

#include "ah_device.hpp"
#include "ah_kernels.hpp"
#include "ah_random.hpp"
#include "../../include/ah.h"

namespace ah {
namespace {

// Eight consecutive elements of a row, of which `left` exist: whole ones in 16-byte accesses at any alignment.
template <typename T>
struct Eight {
    T e[8];
    __device__ __forceinline__ void load(const T* p, int64_t left) {
        if (left >= 8) {
            __builtin_memcpy(e, p, sizeof(e));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = j < left ? p[j] : T(0);
        }
    }
    __device__ __forceinline__ void store(T* p, int64_t left) const {
        if (left >= 8) {
            __builtin_memcpy(p, e, sizeof(e));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < left) p[j] = e[j];
        }
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (sizeof(T) == 4)
            return e[j];
        else
            return __uint_as_float((uint32_t)e[j] << 16);
    }
    __device__ __forceinline__ void set(int j, float v) {
        if constexpr (sizeof(T) == 4)
            e[j] = v;
        else
            e[j] = __builtin_bit_cast(uint16_t, (__bf16)v);
    }
};

struct Args {
    int64_t items, per, n, xs, rs, os;  // items of eight columns, per row
    uint32_t mul, shift;                // v / per = v * mul >> shift for v < 2^31
    Dropout d;
};

// HBM-bound: bfloat16 with a residual, 32768 x 4096: 159 us, 5.07 TB/s (805 MB); an element a thread, with a Philox call
// for each, took 427.  One call serves eight columns, which are one 16-byte access.
// A thread has U items, 256 apart, all read before the first is written (so an output may be its input).
template <typename T, bool RES, int U>
__global__ __launch_bounds__(256) void dropout_kernel(const T* x, const T* res, T* out, Args a) {
    const uint64_t step = a.d.t ? step_of_call(a.d) : 0;
    for (int64_t i0 = (int64_t)blockIdx.x * 256 * U; i0 < a.items; i0 += (int64_t)gridDim.x * 256 * U) {
        const int64_t r0 = i0 / a.per;
        const uint32_t c0 = (uint32_t)(i0 - r0 * a.per);
        Eight<T> v[U], s[RES ? U : 1];
        int64_t row[U];
        uint32_t c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t w = c0 + u * 256 + threadIdx.x, q = (uint32_t)(((uint64_t)w * a.mul) >> a.shift);
            row[u] = r0 + q;
            c[u] = w - q * (uint32_t)a.per;
            if (i0 + u * 256 + threadIdx.x < a.items) {
                v[u].load(x + row[u] * a.xs + (int64_t)c[u] * 8, a.n - (int64_t)c[u] * 8);
                if constexpr (RES) s[u].load(res + row[u] * a.rs + (int64_t)c[u] * 8, a.n - (int64_t)c[u] * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u * 256 + threadIdx.x >= a.items) continue;
            const Philox k = philox(a.d, step, (uint32_t)row[u], c[u]);
            Eight<T> y;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float f = k.at(j) >= a.d.t ? v[u].get(j) * a.d.factor : 0.0f;
                if constexpr (RES) f += s[u].get(j);
                y.set(j, f);
            }
            y.store(out + row[u] * a.os + (int64_t)c[u] * 8, a.n - (int64_t)c[u] * 8);
        }
    }
}

}  // namespace

hipError_t launch_dropout(const void* x, int32_t dtype, int64_t rows, int64_t n, int64_t xs, const Dropout& d,
                          const void* res, int64_t rs, void* out, int64_t os, hipStream_t stream) {
    const int64_t per = (n + 7) / 8;
    Args a{rows * per, per, n, xs, rs, os, 0, 0, d};
    int l = 0;
    while (((int64_t)1 << l) < per) ++l;
    a.shift = 31 + l;
    a.mul = (uint32_t)((((uint64_t)1 << (31 + l)) + per - 1) / per);
    auto go = [&](auto* p, auto res_c, auto u_c) {
        typedef std::remove_const_t<std::remove_pointer_t<decltype(p)>> T;
        constexpr bool R = decltype(res_c)::value;
        constexpr int U = decltype(u_c)::value;
        const int64_t wgs = (a.items + 256 * U - 1) / (256 * U);
        hipLaunchKernelGGL((dropout_kernel<T, R, U>), dim3((uint32_t)(wgs < (1 << 20) ? wgs : 1 << 20)), dim3(256), 0,
                           stream, p, static_cast<const T*>(res), static_cast<T*>(out), a);
        return hipGetLastError();
    };
    auto sized = [&](auto* p, auto u_c) {
        return res ? go(p, std::true_type(), u_c) : go(p, std::false_type(), u_c);
    };
    // Few items: one a thread, so that they spread over the chip (16 x 1536: 2.8 us on the GPU, a launch's latency).
    auto typed = [&](auto* p) {
        return a.items < 256 * 1024 ? sized(p, std::integral_constant<int, 1>())
                                    : sized(p, std::integral_constant<int, 4>());
    };
    return dtype == AH_F32 ? typed(static_cast<const float*>(x)) : typed(static_cast<const uint16_t*>(x));
}

}  // namespace ah
