// Distillation of a student's scores from a teacher's best (ids, scores), loss and
// gradient in one call.  Per row, with p = softmax(t / tau) over the teacher's
// entries and q = softmax(z / tau) over all V student scores:
//   loss = tau^2 sum_j p_j (log p_j - log q[id_j])
//   d loss / d z_v = tau (q_v - sum of p_j over the entries with id_j = v)
// A row without an entry has loss 0 and gradient 0.  Sums and maxima are float32;
// only the gradient is rounded, once, to the scores' type.
#include "ah_device.hpp"
#include "ah_kernels.hpp"
#include "../../include/ah.h"

namespace ah {
namespace {

constexpr int kDT = 512, kDW = kDT / 64;
constexpr float kLog2e = 1.44269504088896340736f;

template <typename T>
__device__ __forceinline__ float score_f32(T v) {
    if constexpr (sizeof(T) == 4)
        return v;
    else
        return __uint_as_float((uint32_t)v << 16);
}
template <typename T>
__device__ __forceinline__ T score_bits(float v) {
    if constexpr (sizeof(T) == 4)
        return v;
    else
        return __builtin_bit_cast(uint16_t, (__bf16)v);
}

struct DistillArgs {
    const void* z;
    int64_t n, V, zs;
    const int32_t* ids;
    const float* t;
    int32_t k;
    float tau, inv_tau;
    const float* weight;
    float* loss;
    void* grad;
    int64_t gs;
};

struct DistillShared {
    float red[kDW];
    float p[AH_MAX_R];   // teacher's probabilities
    float z[AH_MAX_R];   // student's scores at the entries
    int32_t id[AH_MAX_R];
};

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}
__device__ __forceinline__ float wg_sum(float v, float* red) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int w = 1; w < kDW; ++w) s += red[w];
    return s;
}
__device__ __forceinline__ float wg_max(float v, float* red) {
    v = wave_max(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int w = 1; w < kDW; ++w) s = fmaxf(s, red[w]);
    return s;
}

// e^(x) with x already in units of ln 2
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// A maximum to subtract: 0 where every score so far is -inf (or none was seen).
__device__ __forceinline__ float top(float m) { return m == -INFINITY ? 0.0f : m; }

// One workgroup per row, the row read twice.
template <typename T>
__global__ __launch_bounds__(kDT) void distill_row_kernel(DistillArgs a) {
    __shared__ DistillShared sh;
    constexpr int NV = 16 / sizeof(T);
    const int tid = threadIdx.x;
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        const T* z = static_cast<const T*>(a.z) + row * a.zs;
        T* gr = a.grad ? static_cast<T*>(a.grad) + row * a.gs : nullptr;
        const int32_t* ids = a.ids + row * a.k;
        const float* ts = a.t + row * a.k;
        // teacher: entries with an id of the student and a score above -inf
        float tm = -INFINITY;
        bool any = false;
        __syncthreads();
        for (int32_t j = tid; j < a.k; j += kDT) {
            const int32_t id = ids[j];
            const float t = ts[j];
            const bool ok = id >= 0 && id < a.V && !(t == -INFINITY);
            sh.id[j] = ok ? id : -1;
            sh.p[j] = t;
            sh.z[j] = ok ? score_f32(z[id]) : 0.0f;
            if (ok) tm = fmaxf(tm, t);
            any |= ok;
        }
        const bool some = __syncthreads_or(any);
        if (!some) {
            if (tid == 0) a.loss[row] = 0.0f;
            if (gr)
                for (int64_t v = tid; v < a.V; v += kDT) gr[v] = 0;
            continue;
        }
        tm = wg_max(tm, sh.red);
        float ps = 0.0f;
        for (int32_t j = tid; j < a.k; j += kDT)
            if (sh.id[j] >= 0) ps += expf((sh.p[j] - tm) * a.inv_tau);
        ps = wg_sum(ps, sh.red);
        // student: running maximum and sum of 2^((z - max) c).  The difference comes before the
        // factor, so that neither the type's lowest value nor a small tau overflows
        const float c = a.inv_tau * kLog2e;
        float m = -INFINITY, s = 0.0f;
        const int64_t full = a.V / NV;
        for (int64_t i = tid; i < full; i += kDT) {
            T e[NV];
            __builtin_memcpy(e, z + i * NV, 16);
            float mx = m;
#pragma unroll
            for (int r = 0; r < NV; ++r) mx = fmaxf(mx, score_f32(e[r]));
            const float b = top(mx);
            s *= exp2_fast((m - b) * c);
#pragma unroll
            for (int r = 0; r < NV; ++r) s += exp2_fast((score_f32(e[r]) - b) * c);
            m = mx;
        }
        for (int64_t v = full * NV + tid; v < a.V; v += kDT) {
            const float x = score_f32(z[v]), mx = fmaxf(m, x), b = top(mx);
            s = s * exp2_fast((m - b) * c) + exp2_fast((x - b) * c);
            m = mx;
        }
        const float M = top(wg_max(m, sh.red));
        s = wg_sum(s * exp2_fast((m - M) * c), sh.red);
        const float ls = logf(s), lt = logf(ps);
        float l = 0.0f;
        for (int32_t j = tid; j < a.k; j += kDT) {
            if (sh.id[j] < 0) continue;
            const float lp = (sh.p[j] - tm) * a.inv_tau - lt, p = expf(lp);
            if (!(p == 0.0f)) l += p * (lp - (sh.z[j] == -INFINITY ? -INFINITY : (sh.z[j] - M) * a.inv_tau - ls));
            sh.p[j] = p;
        }
        l = wg_sum(l, sh.red);  // its barriers also publish p
        if (tid == 0) a.loss[row] = l * a.tau * a.tau;
        if (!gr) continue;
        const float wt = (a.weight ? a.weight[row] : 1.0f) * a.tau, inv = s > 0.0f || s != s ? 1.0f / s : 0.0f;
        for (int64_t i = tid; i < full; i += kDT) {
            T e[NV];
            __builtin_memcpy(e, z + i * NV, 16);
#pragma unroll
            for (int r = 0; r < NV; ++r) e[r] = score_bits<T>(wt * (exp2_fast((score_f32(e[r]) - M) * c) * inv));
            __builtin_memcpy(gr + i * NV, e, 16);
        }
        for (int64_t v = full * NV + tid; v < a.V; v += kDT)
            gr[v] = score_bits<T>(wt * (exp2_fast((score_f32(z[v]) - M) * c) * inv));
        __syncthreads();
        for (int32_t j = tid; j < a.k; j += kDT) {
            const int32_t id = sh.id[j];
            if (id < 0) continue;
            float p = 0.0f;  // entries that repeat an id add up, each writing the same value
            for (int32_t i = 0; i < a.k; ++i) p += sh.id[i] == id ? sh.p[i] : 0.0f;
            gr[id] = score_bits<T>(wt * (exp2_fast((sh.z[j] - M) * c) * inv - p));
        }
    }
}

}  // namespace

size_t distill_workspace_bytes(int64_t, int64_t) { return 0; }

hipError_t launch_distill(const void* logits, int32_t dtype, int64_t n, int64_t V, int64_t stride, const int32_t* ids,
                          const float* scores, int32_t k, float tau, const float* weight, float* loss, void* grad,
                          int64_t grad_stride, void*, hipStream_t stream) {
    DistillArgs a{logits, n, V, stride, ids, scores, k, tau, 1.0f / tau, weight, loss, grad, grad_stride};
    const uint32_t wgs = (uint32_t)(n < (1 << 20) ? n : 1 << 20);
    if (dtype == AH_F32)
        hipLaunchKernelGGL(distill_row_kernel<float>, dim3(wgs), dim3(kDT), 0, stream, a);
    else
        hipLaunchKernelGGL(distill_row_kernel<uint16_t>, dim3(wgs), dim3(kDT), 0, stream, a);
    return hipGetLastError();
}

}  // namespace ah
