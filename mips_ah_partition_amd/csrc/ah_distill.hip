// Distillation of a student's scores from a teacher's best (ids, scores), loss and
// gradient in one call.  Per row, with p = softmax(t / tau) over the teacher's
// entries and q = softmax(z / tau) over all V student scores:
//   loss = tau^2 sum_j p_j (log p_j - log q[id_j])
//   d loss / d z_v = tau (q_v - sum of p_j over the entries with id_j = v)
// A row without an entry has loss 0 and gradient 0.  Sums and maxima are float32;
// only the gradient is rounded, once, to the scores' type.
//
// HBM-bound: the scores in, the gradient out.
//   Many rows of at most 128 KB   one workgroup per row, which is kept in registers between
//                                 the sum and the gradient: every byte moves once
//   few rows, or longer ones      a row is cut into slices, one workgroup each, and the call into two
//                                 launches: maximum and sum of each slice, then the gradient;
//                                 rows go in groups whose scores stay in the last-level cache
//                                 between the two
// Measured: bfloat16 4096 x 65,536 in 207 us (5.2 TB/s; a copy reaches 5.0); float32 1000 x 4000 in
// 12.9 us for the call; bfloat16 3 x 250,001 in 3.6 + 5.9 us on the GPU (49 us with a workgroup a row).
// 1024 threads a row instead of 512: 262 us for the first.
#include "ah_device.hpp"
#include "ah_kernels.hpp"
#include "../../include/ah.h"

namespace ah {
namespace {

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
    float c;  // log2(e) / tau, rounded once: exponents scale by it, so its error grows with them
    const float* weight;
    float* loss;
    void* grad;
    int64_t gs;
    float* part;     // split rows: [n][slices][2] maximum and sum
    float* entries;  // split rows: [n][k] the student's scores at the entries
    int32_t slices;
    int64_t slice;   // scores of a slice (a multiple of 8)
};

struct Teacher {  // in LDS, 128 + 12 bytes an entry, their number rounded up to four
    float* red;
    float* p;     // teacher's scores, then probabilities
    float* z;     // student's scores at the entries
    int32_t* id;  // -1: no entry
};
extern __shared__ __align__(16) float teacher_lds[];
__device__ __forceinline__ Teacher teacher(int32_t k) {
    const int32_t n = (k + 3) & ~3;
    return Teacher{teacher_lds, teacher_lds + 32, teacher_lds + 32 + n, reinterpret_cast<int32_t*>(teacher_lds + 32 + 2 * n)};
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}
// Sums and maxima over a workgroup, in a fixed order; red: two words a wave.
template <int NT>
__device__ __forceinline__ float wg_sum(float v, float* red) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) s += red[w];
    return s;
}
template <int NT>
__device__ __forceinline__ void wg_sum2(float& a, float& b, float* red) {
    const float u = wave_sum(a), v = wave_sum(b);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        red[threadIdx.x >> 6] = u;
        red[NT / 64 + (threadIdx.x >> 6)] = v;
    }
    __syncthreads();
    a = red[0];
    b = red[NT / 64];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) {
        a += red[w];
        b += red[NT / 64 + w];
    }
}
template <int NT>
__device__ __forceinline__ void wg_max2(float& a, float& b, float* red) {
    const float u = wave_max(a), v = wave_max(b);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        red[threadIdx.x >> 6] = u;
        red[NT / 64 + (threadIdx.x >> 6)] = v;
    }
    __syncthreads();
    a = red[0];
    b = red[NT / 64];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) {
        a = fmaxf(a, red[w]);
        b = fmaxf(b, red[NT / 64 + w]);
    }
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// A maximum to subtract: 0 where every score so far is -inf (or none was seen).
__device__ __forceinline__ float top(float m) { return m == -INFINITY ? 0.0f : m; }

template <typename T>
struct Chunk {  // 16 bytes of scores, kept packed
    static constexpr int N = 16 / sizeof(T);
    v4i raw;
    __device__ __forceinline__ void load(const T* p) { __builtin_memcpy(&raw, p, 16); }
    __device__ __forceinline__ void floats(float* f) const {
        T e[N];
        __builtin_memcpy(e, &raw, 16);
#pragma unroll
        for (int r = 0; r < N; ++r) f[r] = score_f32(e[r]);
    }
    // What was unpacked so far is forgotten: the next pass unpacks again, instead of holding floats between.
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(raw)); }
    __device__ __forceinline__ float max(float m) const {
        float f[N];
        floats(f);
#pragma unroll
        for (int r = 0; r < N; ++r) m = fmaxf(m, f[r]);
        return m;
    }
    // sum of 2^((z - M) c).  The difference comes before the factor, so that neither the type's
    // lowest value nor a small tau overflows
    __device__ __forceinline__ float sum(float M, float c) const {
        float f[N], s = 0.0f;
        floats(f);
#pragma unroll
        for (int r = 0; r < N; ++r) s += exp2_fast((f[r] - M) * c);
        return s;
    }
    __device__ __forceinline__ void grad(float M, float c, float scale, T* o) const {
        float f[N];
        T g[N];
        floats(f);
#pragma unroll
        for (int r = 0; r < N; ++r) g[r] = score_bits<T>(scale * exp2_fast((f[r] - M) * c));
        __builtin_memcpy(o, g, 16);
    }
};
// Zeros to gr[v0, v1).
template <typename T, int NT>
__device__ __forceinline__ void clear_grads(T* gr, int64_t v0, int64_t v1) {
    constexpr int N = Chunk<T>::N;
    const v4i zero = {0, 0, 0, 0};
    const int64_t full = (v1 - v0) / N;
    for (int64_t i = threadIdx.x; i < full; i += NT) __builtin_memcpy(gr + v0 + i * N, &zero, 16);
    for (int64_t v = v0 + full * N + threadIdx.x; v < v1; v += NT) gr[v] = 0;
}

// The teacher's entries of a row into LDS (an entry has an id of the student and a score above -inf);
// z(j, id): the student's score of entry j.  Returns whether there is one (after a barrier), and in *tm the
// thread's largest.
template <int NT, typename F>
__device__ __forceinline__ bool take_entries(const DistillArgs& a, int64_t row, const Teacher& sh, float* tm,
                                             const F& z) {
    const int32_t* ids = a.ids + row * a.k;
    const float* ts = a.t + row * a.k;
    bool any = false;
    *tm = -INFINITY;
    for (int32_t j = threadIdx.x; j < ((a.k + 3) & ~3); j += NT) {
        const int32_t id = j < a.k ? ids[j] : -1;
        const float t = j < a.k ? ts[j] : 0.0f;
        const bool ok = id >= 0 && id < a.V && !(t == -INFINITY);
        sh.id[j] = ok ? id : -1;
        sh.p[j] = t;
        sh.z[j] = ok ? z(j, id) : 0.0f;
        if (ok) *tm = fmaxf(*tm, t);
        any |= ok;
    }
    return __syncthreads_or(any);
}
// The thread's part of the teacher's sum, tm its largest score.
template <int NT>
__device__ __forceinline__ float entry_sum(const DistillArgs& a, const Teacher& sh, float tm) {
    float s = 0.0f;
    for (int32_t j = threadIdx.x; j < a.k; j += NT)
        if (sh.id[j] >= 0) s += expf((sh.p[j] - tm) * a.inv_tau);
    return s;
}
// Loss of a row, by every thread; sh.p becomes the probabilities (published by its barriers).  M, s: the
// student's maximum and sum; tm, ts: the teacher's.
template <int NT>
__device__ __forceinline__ float row_loss(const DistillArgs& a, const Teacher& sh, float M, float s, float tm,
                                          float ts) {
    const float lt = logf(ts), ls = logf(s);
    float l = 0.0f;
    for (int32_t j = threadIdx.x; j < a.k; j += NT) {
        if (sh.id[j] < 0) continue;
        const float lp = (sh.p[j] - tm) * a.inv_tau - lt, p = expf(lp);
        if (!(p == 0.0f)) l += p * (lp - (sh.z[j] == -INFINITY ? -INFINITY : (sh.z[j] - M) * a.inv_tau - ls));
        sh.p[j] = p;
    }
    return wg_sum<NT>(l, sh.red) * a.tau * a.tau;
}
// Gradients at the entries with an id in [v0, v1), over what was written there before.
template <typename T, int NT>
__device__ __forceinline__ void entry_grads(const DistillArgs& a, const Teacher& sh, T* gr, int64_t v0, int64_t v1,
                                            float M, float c, float inv, float wt) {
    __syncthreads();
    for (int32_t j = threadIdx.x; j < a.k; j += NT) {
        const int32_t id = sh.id[j];
        if (id < 0 || id < v0 || id >= v1) continue;
        float p = 0.0f;  // entries that repeat an id add up, each writing the same value
#pragma unroll 4
        for (int32_t i = 0; i < (a.k + 3) >> 2; ++i) {
            const v4i d = reinterpret_cast<const v4i*>(sh.id)[i];
            const v4f q = reinterpret_cast<const v4f*>(sh.p)[i];
#pragma unroll
            for (int e = 0; e < 4; ++e) p += d[e] == id ? q[e] : 0.0f;
        }
        gr[id] = score_bits<T>(wt * (exp2_fast((sh.z[j] - M) * c) * inv - p));
    }
}
__device__ __forceinline__ float inverse(float s) { return s == 0.0f ? 0.0f : 1.0f / s; }  // all -inf: q = 0

// One workgroup per row, KEEP chunks of it in each thread.
template <typename T, int NT, int KEEP>
__global__ __launch_bounds__(NT, 4) void distill_row_kernel(DistillArgs a) {
    typedef Chunk<T> C;
    const Teacher sh = teacher(a.k);
    const int tid = threadIdx.x;
    const int32_t full = (int32_t)(a.V / C::N), rest = (int32_t)(a.V % C::N);
    const int64_t row = blockIdx.x;
    const T* z = static_cast<const T*>(a.z) + row * a.zs;
    T* gr = a.grad ? static_cast<T*>(a.grad) + row * a.gs : nullptr;
    C x[KEEP];  // threads past the row's end repeat its last whole chunk and leave it out of the sum
    float last = -INFINITY;  // of the scores past the last whole chunk
#pragma unroll
    for (int u = 0; u < KEEP; ++u) x[u].raw = v4i{0, 0, 0, 0};
    if (full > 0) {
#pragma unroll
        for (int u = 0; u < KEEP; ++u)
            x[u].load(reinterpret_cast<const T*>(reinterpret_cast<const char*>(z) +
                                                 (uint32_t)(u * NT + tid < full ? u * NT + tid : full - 1) * 16u));
    }
    if (tid < rest) last = score_f32(z[a.V - rest + tid]);
    float tm;
    const bool some = take_entries<NT>(a, row, sh, &tm, [&](int32_t, int32_t id) { return score_f32(z[id]); });
    if (!some) {
        if (tid == 0) a.loss[row] = 0.0f;
        if (gr) clear_grads<T, NT>(gr, 0, a.V);
        return;
    }
    float m = last;
    if (full > 0) {
#pragma unroll
        for (int u = 0; u < KEEP; ++u) {
            m = x[u].max(m);
            x[u].forget();
        }
    }
    wg_max2<NT>(m, tm, sh.red);
    const float c = a.c, M = top(m);
    float s = exp2_fast((last - M) * c), ts = entry_sum<NT>(a, sh, tm);
#pragma unroll
    for (int u = 0; u < KEEP; ++u) {
        const float e = x[u].sum(M, c);
        if (u * NT + tid < full) s += e;
        x[u].forget();
        __builtin_amdgcn_sched_barrier(0);  // one chunk's floats at a time
    }
    wg_sum2<NT>(s, ts, sh.red);
    const float l = row_loss<NT>(a, sh, M, s, tm, ts);
    if (tid == 0) a.loss[row] = l;
    if (gr) {
        const float wt = (a.weight ? a.weight[row] : 1.0f) * a.tau, inv = inverse(s);
        int at = threadIdx.x;  // taken as new: no offset of the loads is held until here
        asm volatile("" : "+v"(at));
#pragma unroll
        for (int u = 0; u < KEEP; ++u) {
            if (u * NT + at < full)
                x[u].grad(M, c, wt * inv,
                          reinterpret_cast<T*>(reinterpret_cast<char*>(gr) + (uint32_t)(u * NT + at) * 16u));
            __builtin_amdgcn_sched_barrier(0);
        }
        if (tid < rest) gr[a.V - rest + tid] = score_bits<T>(wt * inv * exp2_fast((last - M) * c));
        entry_grads<T, NT>(a, sh, gr, 0, a.V, M, c, inv, wt);
    }
}

// Split rows, first launch: maximum and sum of a slice (a wave's lanes, then waves, then slices are joined in a
// fixed order), and the student's scores at the entries (the gradient may overwrite them).
constexpr int kST = 256;
template <typename T>
__global__ __launch_bounds__(kST) void distill_part_kernel(DistillArgs a) {
    typedef Chunk<T> C;
    __shared__ float red[2 * kST / 64];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / (uint32_t)a.slices, sl = blockIdx.x % (uint32_t)a.slices;
    const int64_t v0 = sl * a.slice, v1 = v0 + a.slice < a.V ? v0 + a.slice : a.V;
    const T* z = static_cast<const T*>(a.z) + row * a.zs;
    const float c = a.c;
    const int64_t full = (v1 - v0) / C::N;
    float m = -INFINITY, s = 0.0f;
    constexpr int U = 4;
    for (int64_t i = tid; i < full; i += U * kST) {
        C x[U];
        float mx = m;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * kST < full) x[u].load(z + v0 + (i + u * kST) * C::N);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * kST < full) mx = x[u].max(mx);
        const float b = top(mx);
        s *= exp2_fast((m - b) * c);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * kST < full) s += x[u].sum(b, c);
        m = mx;
    }
    for (int64_t v = v0 + full * C::N + tid; v < v1; v += kST) {
        const float x = score_f32(z[v]), mx = fmaxf(m, x), b = top(mx);
        s = s * exp2_fast((m - b) * c) + exp2_fast((x - b) * c);
        m = mx;
    }
    float M = m, none = m;
    wg_max2<kST>(M, none, red);
    s = wg_sum<kST>(s * exp2_fast((m - top(M)) * c), red);
    if (tid == 0) {
        a.part[blockIdx.x * 2] = M;
        a.part[blockIdx.x * 2 + 1] = s;
    }
    if (sl == 0)
        for (int32_t j = tid; j < a.k; j += kST) {
            const int32_t id = a.ids[row * a.k + j];
            a.entries[row * a.k + j] = id >= 0 && id < a.V ? score_f32(z[id]) : 0.0f;
        }
}

// Second launch: the row's maximum and sum from its slices', the loss (by the first), the slice's gradient.
template <typename T>
__global__ __launch_bounds__(kST) void distill_grad_kernel(DistillArgs a) {
    typedef Chunk<T> C;
    const Teacher sh = teacher(a.k);
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / (uint32_t)a.slices, sl = blockIdx.x % (uint32_t)a.slices;
    const int64_t v0 = sl * a.slice, v1 = v0 + a.slice < a.V ? v0 + a.slice : a.V;
    const T* z = static_cast<const T*>(a.z) + row * a.zs;
    T* gr = a.grad ? static_cast<T*>(a.grad) + row * a.gs : nullptr;
    float tm;
    const bool some = take_entries<kST>(a, row, sh, &tm, [&](int32_t j, int32_t) { return a.entries[row * a.k + j]; });
    if (!some) {
        if (tid == 0 && sl == 0) a.loss[row] = 0.0f;
        if (gr) clear_grads<T, kST>(gr, v0, v1);
        return;
    }
    const float c = a.c;
    const float* part = a.part + row * a.slices * 2;
    float m = -INFINITY, s = 0.0f;
    for (int32_t i = tid; i < a.slices; i += kST) m = fmaxf(m, part[2 * i]);
    wg_max2<kST>(m, tm, sh.red);
    const float M = top(m);
    for (int32_t i = tid; i < a.slices; i += kST) {
        const float pm = part[2 * i], ps = part[2 * i + 1];
        s += pm == -INFINITY ? ps : ps * exp2_fast((pm - M) * c);
    }
    float ts = entry_sum<kST>(a, sh, tm);
    wg_sum2<kST>(s, ts, sh.red);
    const float l = row_loss<kST>(a, sh, M, s, tm, ts);
    if (tid == 0 && sl == 0) a.loss[row] = l;
    if (!gr) return;
    const float wt = (a.weight ? a.weight[row] : 1.0f) * a.tau, inv = inverse(s);
    const int64_t full = (v1 - v0) / C::N;
    constexpr int U = 4;
    for (int64_t i = tid; i < full; i += U * kST) {
        C x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * kST < full) x[u].load(z + v0 + (i + u * kST) * C::N);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * kST < full) x[u].grad(M, c, wt * inv, gr + v0 + (i + u * kST) * C::N);
    }
    for (int64_t v = v0 + full * C::N + tid; v < v1; v += kST)
        gr[v] = score_bits<T>(wt * inv * exp2_fast((score_f32(z[v]) - M) * c));
    entry_grads<T, kST>(a, sh, gr, v0, v1, M, c, inv, wt);
}

constexpr int64_t kRowBytes = 128 << 10;    // kept by a workgroup of 512 threads, 16 chunks each, two workgroups a CU
constexpr int64_t kFewRows = 128;           // below this a workgroup per row leaves CUs idle
constexpr int64_t kCacheBytes = 96 << 20;   // scores of a group of split rows
constexpr int64_t kSplitWgs = 1024;

bool split_rows(int64_t n, int64_t row_bytes) {
    return row_bytes > kRowBytes || (n < kFewRows && row_bytes > (16 << 10));
}
// Slices of a row: enough workgroups for the chip, pieces of 4 KB at least and 128 KB at most.
void cut(int64_t n, int64_t V, int64_t elem, int32_t* slices, int64_t* slice) {
    const int64_t bytes = V * elem;
    int64_t s = (kSplitWgs + n - 1) / n;
    if (s > bytes / 4096) s = bytes / 4096;
    if (s < (bytes + (128 << 10) - 1) / (128 << 10)) s = (bytes + (128 << 10) - 1) / (128 << 10);
    *slice = ((V + s - 1) / s + 7) / 8 * 8;
    *slices = (int32_t)((V + *slice - 1) / *slice);
}

// The call's next rows, after the first a.n.
template <typename T>
void next_rows(DistillArgs& a) {
    a.z = static_cast<const T*>(a.z) + a.n * a.zs;
    a.ids += a.n * a.k;
    a.t += a.n * a.k;
    if (a.weight) a.weight += a.n;
    a.loss += a.n;
    if (a.grad) a.grad = static_cast<T*>(a.grad) + a.n * a.gs;
}

template <typename T>
hipError_t launch(DistillArgs a, void* ws, hipStream_t stream) {
    const int64_t bytes = a.V * (int64_t)sizeof(T), all = a.n;
    const uint32_t lds = 128 + 12 * (((uint32_t)a.k + 3) & ~3u);
    if (!split_rows(a.n, bytes)) {
        const int nt = bytes <= (16 << 10) + 15 ? 256 : 512;
        const int64_t most = kMaxGridItems / nt;  // rows of one launch
        for (int64_t r = 0; r < all; r += most) {
            a.n = all - r < most ? all - r : most;
            const dim3 grid((uint32_t)a.n);
            if (nt == 256)
                hipLaunchKernelGGL((distill_row_kernel<T, 256, 4>), grid, dim3(256), lds, stream, a);
            else if (bytes <= (64 << 10) + 15)
                hipLaunchKernelGGL((distill_row_kernel<T, 512, 8>), grid, dim3(512), lds, stream, a);
            else
                hipLaunchKernelGGL((distill_row_kernel<T, 512, 16>), grid, dim3(512), lds, stream, a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            next_rows<T>(a);
        }
        return hipSuccess;
    }
    const int64_t group = kCacheBytes / bytes < 1 ? 1 : kCacheBytes / bytes;
    for (int64_t r = 0; r < all; r += group) {
        a.n = all - r < group ? all - r : group;
        cut(a.n, a.V, sizeof(T), &a.slices, &a.slice);
        a.entries = static_cast<float*>(ws);
        a.part = a.entries + a.n * a.k;
        const dim3 grid((uint32_t)(a.n * a.slices));
        hipLaunchKernelGGL(distill_part_kernel<T>, grid, dim3(kST), 0, stream, a);
        hipLaunchKernelGGL(distill_grad_kernel<T>, grid, dim3(kST), lds, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        next_rows<T>(a);
    }
    return hipSuccess;
}

}  // namespace

size_t distill_workspace_bytes(int64_t n, int64_t V, int32_t k) {
    size_t need = 0;
    for (int64_t elem = 2; elem <= 4; elem += 2) {
        if (n < 1 || !split_rows(n, V * elem)) continue;
        const int64_t group = kCacheBytes / (V * elem) < 1 ? 1 : kCacheBytes / (V * elem);
        for (int64_t rows : {n < group ? n : group, n % group}) {  // the groups, and the last one
            if (rows < 1) continue;
            int32_t slices;
            int64_t slice;
            cut(rows, V, elem, &slices, &slice);
            const size_t b = (size_t)rows * (2 * (size_t)slices + (size_t)k) * sizeof(float);
            need = b > need ? b : need;
        }
    }
    return need;
}

hipError_t launch_distill(const void* logits, int32_t dtype, int64_t n, int64_t V, int64_t stride, const int32_t* ids,
                          const float* scores, int32_t k, float tau, const float* weight, float* loss, void* grad,
                          int64_t grad_stride, void* ws, hipStream_t stream) {
    const float c = (float)(1.44269504088896340736 / (double)tau);
    const DistillArgs a{logits, n, V, stride, ids, scores, k, tau, 1.0f / tau, c, weight, loss, grad, grad_stride,
                        nullptr, nullptr, 0, 0};
    return dtype == AH_F32 ? launch<float>(a, ws, stream) : launch<uint16_t>(a, ws, stream);
}

}  // namespace ah
