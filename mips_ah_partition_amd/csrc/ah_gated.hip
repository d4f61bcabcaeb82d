// Gated feed-forward by leaf: h = keep(act(W_gate x) * (W_up x)) and its backward pass up to the two
// projections' gradients.
#include "ah_device.hpp"
#include "ah_kernels.hpp"
#include "ah_gating.hpp"
#include "ah_simple.hpp"
#include "../../include/ah.h"

namespace ah {
namespace {

__device__ __forceinline__ float f32_of(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t bits_of(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// A row tile of a leaf (z < L), or of the rows of no leaf (z == L): grouped rows [p0, p1).
__device__ __forceinline__ int64_t start_of(const GatedProblem& g, int32_t l) {
    const int64_t o = g.offsets ? g.offsets[l] : l ? g.slots : 0;
    return o < 0 ? 0 : o > g.slots ? g.slots : o;
}
__device__ __forceinline__ int64_t slot_at(const GatedProblem& g, int64_t p) {
    if (!g.order) return p;
    const int32_t s = g.order[p];
    return s >= 0 && s < g.slots ? s : -1;
}

template <class Tile, class Zero>
__device__ __forceinline__ void each_tile(const GatedProblem& g, Tile tile, Zero zero) {
    if ((int32_t)blockIdx.z == g.L) {
        const int64_t head = start_of(g, 0), tail = start_of(g, g.L);
        for (int64_t p = blockIdx.y; p < head + g.slots - tail; p += gridDim.y) {
            const int64_t s = slot_at(g, p < head ? p : tail + p - head);
            if (s >= 0) zero(s);
        }
        return;
    }
    const int64_t a = start_of(g, blockIdx.z), b = start_of(g, blockIdx.z + 1);
    for (int64_t p = a + (int64_t)blockIdx.y * 64; p < b; p += (int64_t)gridDim.y * 64) tile(p, b);
}

__global__ __launch_bounds__(256) void gated_kernel(GatedProblem g, Dropout d, int act, uint16_t* pre, void* out,
                                                    int out_f32) {
    const uint64_t step = d.t ? step_of_call(d) : 0;
    const int64_t j0 = (int64_t)blockIdx.x * 64;
    auto put = [&](int64_t s, int64_t j, float h, float a, float b) {
        if (out_f32)
            static_cast<float*>(out)[s * g.n + j] = h;
        else
            static_cast<uint16_t*>(out)[s * g.n + j] = bits_of(h);
        if (pre) {
            pre[s * 2 * g.n + j] = bits_of(a);
            pre[s * 2 * g.n + g.n + j] = bits_of(b);
        }
    };
    each_tile(
        g,
        [&](int64_t p0, int64_t p1) {
            const uint16_t* x = static_cast<const uint16_t*>(g.q);
            const uint16_t* w = static_cast<const uint16_t*>(g.w) + (int64_t)blockIdx.z * 2 * g.n * g.k;
            simple_tile<2>(
                g.k,
                [&](int r, int64_t t) {
                    const int64_t s = p0 + r < p1 ? slot_at(g, p0 + r) : -1;
                    return s < 0 ? 0.0f : f32_of(x[s / g.fan * g.q_stride + t]);
                },
                [&](int h, int c, int64_t t) {
                    return j0 + c < g.n ? f32_of(w[((int64_t)h * g.n + j0 + c) * g.k + t]) : 0.0f;
                },
                [&](int r, int c, const float* v) {
                    const int64_t s = p0 + r < p1 ? slot_at(g, p0 + r) : -1, j = j0 + c;
                    if (s < 0 || j >= g.n) return;
                    float h = activate(act, v[0]) * v[1];
                    if (d.t) h = philox(d, step, (uint32_t)s, (uint32_t)(j >> 3)).at(j & 7) >= d.t ? h * d.factor : 0.0f;
                    put(s, j, h, v[0], v[1]);
                });
        },
        [&](int64_t s) {
            for (int64_t j = j0 + threadIdx.x; j < j0 + 64 && j < g.n; j += 256) put(s, j, 0.0f, 0.0f, 0.0f);
        });
}

__global__ __launch_bounds__(256) void gated_grad_kernel(GatedProblem g, Dropout d, int act, const uint16_t* pre,
                                                         uint16_t* dpre, uint16_t* hidden) {
    const uint64_t step = d.t ? step_of_call(d) : 0;
    const int64_t j0 = (int64_t)blockIdx.x * 64;
    auto put = [&](int64_t s, int64_t j, float da, float db, float h) {
        dpre[s * 2 * g.n + j] = bits_of(da);
        dpre[s * 2 * g.n + g.n + j] = bits_of(db);
        if (hidden) hidden[s * g.n + j] = bits_of(h);
    };
    each_tile(
        g,
        [&](int64_t p0, int64_t p1) {
            const uint16_t* dy = static_cast<const uint16_t*>(g.q);
            const uint16_t* w = static_cast<const uint16_t*>(g.w) + (int64_t)blockIdx.z * g.k * g.n;
            simple_tile<1>(
                g.k,
                [&](int r, int64_t t) {
                    const int64_t s = p0 + r < p1 ? slot_at(g, p0 + r) : -1;
                    return s < 0 ? 0.0f : f32_of(dy[s * g.q_stride + t]);
                },
                [&](int, int c, int64_t t) { return j0 + c < g.n ? f32_of(w[t * g.n + j0 + c]) : 0.0f; },
                [&](int r, int c, const float* v) {
                    const int64_t s = p0 + r < p1 ? slot_at(g, p0 + r) : -1, j = j0 + c;
                    if (s < 0 || j >= g.n) return;
                    const float a = f32_of(pre[s * 2 * g.n + j]), b = f32_of(pre[s * 2 * g.n + g.n + j]);
                    const bool keep = !d.t || philox(d, step, (uint32_t)s, (uint32_t)(j >> 3)).at(j & 7) >= d.t;
                    float f, df;
                    activate_grad(act, a, &f, &df);
                    const float dh = v[0] * d.factor;
                    put(s, j, keep ? dh * b * df : 0.0f, keep ? dh * f : 0.0f, keep ? f * b * d.factor : 0.0f);
                });
        },
        [&](int64_t s) {
            for (int64_t j = j0 + threadIdx.x; j < j0 + 64 && j < g.n; j += 256) put(s, j, 0.0f, 0.0f, 0.0f);
        });
}

dim3 grid_of(const GatedProblem& g) {
    const int64_t rows = (g.slots + 63) / 64;
    return dim3((uint32_t)((g.n + 63) / 64), (uint32_t)(rows < 256 ? rows : 256), (uint32_t)(g.L + 1));
}

}  // namespace

hipError_t launch_gated(const GatedProblem& g, const Dropout& d, int32_t act, void* pre, void* out, int32_t out_dtype,
                        hipStream_t stream) {
    hipLaunchKernelGGL(gated_kernel, grid_of(g), dim3(256), 0, stream, g, d, act, static_cast<uint16_t*>(pre), out,
                       out_dtype == AH_F32);
    return hipGetLastError();
}

hipError_t launch_gated_grad(const GatedProblem& g, const Dropout& d, int32_t act, const void* pre, void* dpre,
                             void* hidden, hipStream_t stream) {
    hipLaunchKernelGGL(gated_grad_kernel, grid_of(g), dim3(256), 0, stream, g, d, act,
                       static_cast<const uint16_t*>(pre), static_cast<uint16_t*>(dpre),
                       static_cast<uint16_t*>(hidden));
    return hipGetLastError();
}

}  // namespace ah
