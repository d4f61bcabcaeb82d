// Rows in leaf order: a stable counting sort of (query, leaf) slots by leaf, the
// order in which the grouped products read and write rows.
//
// Slots are cut into slices of 4,096, one workgroup each, and a slice into eight
// consecutive runs, one wave each.  A slot's place is (rows of smaller leaves) +
// (its leaf's slots in earlier slices) + (in earlier waves' runs) + (earlier in
// its run); the last comes from ballots over the bits of the leaf, so the order
// never depends on the order of atomics.  Slots without a leaf form bin L, the last.
// One slice needs one launch; more take a histogram and a scan over slices first.
#include "ah_device.hpp"
#include "ah_kernels.hpp"
#include "../../include/ah.h"

namespace ah {
namespace {

constexpr int kGT = 512, kGW = kGT / 64, kSlice = 4096, kRun = kSlice / kGW;
constexpr int kMaxBins = AH_MAX_ASSIGN_LEAVES + 1;

__device__ __forceinline__ int bin_of(const int32_t* leaves, int64_t i, int32_t L) {
    const int32_t l = leaves[i];
    return l >= 0 && l < L ? l : L;
}

// Histogram of each slice, bin-major: hist[bin * slices + slice].
__global__ __launch_bounds__(kGT) void group_hist_kernel(const int32_t* leaves, int64_t n, int32_t L, int32_t* hist) {
    __shared__ int32_t h[kMaxBins];
    for (int b = threadIdx.x; b <= L; b += kGT) h[b] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * kSlice;
    for (int64_t i = i0 + threadIdx.x; i < i0 + kSlice && i < n; i += kGT) atomicAdd(&h[bin_of(leaves, i, L)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b <= L; b += kGT) hist[(int64_t)b * gridDim.x + blockIdx.x] = h[b];
}

// One wave per bin: exclusive sums over the slices, in place, and the bin's total.
__global__ __launch_bounds__(256) void group_scan_kernel(int32_t* hist, int64_t slices, int32_t bins, int32_t* total) {
    const int32_t b = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (b >= bins) return;
    int32_t* h = hist + (int64_t)b * slices;
    int32_t run = 0;
    for (int64_t s = lane; s - lane < slices; s += 64) {
        const int32_t v = s < slices ? h[s] : 0;
        const int32_t incl = wave_inclusive_sum(v);
        if (s < slices) h[s] = run + incl - v;
        run += __shfl(incl, 63, 64);
    }
    if (lane == 0) total[b] = run;
}

// Places of one slice's slots.  hist, total NULL: the slice is everything.
__global__ __launch_bounds__(kGT) void group_place_kernel(const int32_t* leaves, int64_t n, int32_t L,
                                                          const int32_t* hist, const int32_t* total, int64_t* offsets,
                                                          int32_t* order) {
    __shared__ int32_t cnt[kGW][kMaxBins];
    __shared__ int32_t wave_sum[kGW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, bins = L + 1;
    for (int w = 0; w < kGW; ++w)
        for (int b = tid; b < bins; b += kGT) cnt[w][b] = 0;
    __syncthreads();
    const int64_t r0 = (int64_t)blockIdx.x * kSlice + wave * kRun;
    for (int64_t i = r0 + lane; i < r0 + kRun && i < n; i += 64) atomicAdd(&cnt[wave][bin_of(leaves, i, L)], 1);
    __syncthreads();
    // rows of smaller bins: each thread scans a run of bins
    const int run = (bins + kGT - 1) / kGT, b0 = tid * run, b1 = b0 + run < bins ? b0 + run : bins;
    int32_t sum = 0;
    for (int b = b0; b < b1; ++b) {
        int32_t t = 0;
        if (total) {
            t = total[b];
        } else {
            for (int w = 0; w < kGW; ++w) t += cnt[w][b];
        }
        sum += t;
    }
    const int32_t incl = wave_inclusive_sum(sum);
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    int32_t at = incl - sum;
    for (int w = 0; w < wave; ++w) at += wave_sum[w];
    for (int b = b0; b < b1; ++b) {
        if (blockIdx.x == 0) offsets[b] = at;  // bin L starts where the last leaf ends
        int32_t t = 0, base = at + (hist ? hist[(int64_t)b * gridDim.x + blockIdx.x] : 0);
        for (int w = 0; w < kGW; ++w) {
            const int32_t c = cnt[w][b];
            cnt[w][b] = base;
            base += c;
            t += c;
        }
        at += total ? total[b] : t;
    }
    __syncthreads();
    const int bits = 32 - __builtin_clz(bins);
    for (int64_t i0 = r0; i0 < r0 + kRun && i0 < n; i0 += 64) {
        const int64_t i = i0 + lane;
        const bool in = i < n;
        const int b = in ? bin_of(leaves, i, L) : 0;
        uint64_t same = __ballot(in);
        for (int k = 0; k < bits; ++k) {
            const uint64_t m = __ballot((b >> k) & 1);
            same &= (b >> k) & 1 ? m : ~m;
        }
        const int rank = __popcll(same & lanemask_lt());
        if (in) {
            order[cnt[wave][b] + rank] = (int32_t)i;
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
            if (rank == 0) cnt[wave][b] += __popcll(same);
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

int64_t slices_of(int64_t n) { return (n + kSlice - 1) / kSlice; }

}  // namespace

size_t group_rows_workspace_bytes(int64_t n, int32_t L) {
    const int64_t s = slices_of(n);
    return s > 1 ? (size_t)(s + 1) * (L + 1) * sizeof(int32_t) : 0;
}

hipError_t launch_group_rows(const int32_t* leaves, int64_t n, int32_t L, int64_t* offsets, int32_t* order, void* ws,
                             hipStream_t stream) {
    const int64_t s = slices_of(n);
    if (s <= 1) {
        hipLaunchKernelGGL(group_place_kernel, dim3(1), dim3(kGT), 0, stream, leaves, n, L, nullptr, nullptr, offsets,
                           order);
        return hipGetLastError();
    }
    int32_t* total = static_cast<int32_t*>(ws);
    int32_t* hist = total + L + 1;
    hipLaunchKernelGGL(group_hist_kernel, dim3((uint32_t)s), dim3(kGT), 0, stream, leaves, n, L, hist);
    hipLaunchKernelGGL(group_scan_kernel, dim3((uint32_t)(L + 4) / 4), dim3(256), 0, stream, hist, s, L + 1, total);
    hipLaunchKernelGGL(group_place_kernel, dim3((uint32_t)s), dim3(kGT), 0, stream, leaves, n, L, hist, total, offsets,
                       order);
    return hipGetLastError();
}

}  // namespace ah
