// Rows in leaf order: a stable counting sort of (query, leaf) slots by leaf, the
// order in which the grouped products read and write rows.
//
// Slots are cut into slices, one workgroup each, and a slice into eight consecutive
// runs, one wave each.  A slot's place is (rows of smaller leaves) + (its leaf's slots in
// earlier slices) + (in earlier waves' runs) + (earlier in its run); the last comes
// from ballots over the bits of the leaf, so the order never depends on the order of
// atomics.  Slots without a leaf form bin L, the last.
//   one slice (4,096 slots)          one launch
//   few (slice, leaf) counts         two: the slices' histograms, and the places, where every
//                                    workgroup adds up the histograms for itself
//   else                             three: a scan over the slices, one wave a leaf, between them
// Bound by launches and by the latency of a run's loads, which are all started at once: 32,768
// slots of 64 leaves 5 + 6 us.
#include "ah_device.hpp"
#include "ah_kernels.hpp"
#include "../../include/ah.h"

namespace ah {
namespace {

constexpr int kGT = 512, kGW = kGT / 64, kRounds = 8;  // a run is at most 8 x 64 slots
constexpr int64_t kOneSlice = kGW * kRounds * 64;
constexpr int64_t kDirect = 1 << 16;                   // (slice, bin) counts that every workgroup may add up
constexpr int kMaxBins = AH_MAX_ASSIGN_LEAVES + 1;

__device__ __forceinline__ int bin_of(const int32_t* leaves, int64_t i, int32_t L) {
    const int32_t l = leaves[i];
    return l >= 0 && l < L ? l : L;
}

// Histogram of each slice, hist[bin * bin_step + slice * slice_step].
__global__ __launch_bounds__(kGT) void group_hist_kernel(const int32_t* leaves, int64_t n, int32_t L, int32_t slice,
                                                         int64_t bin_step, int64_t slice_step, int32_t* hist) {
    __shared__ int32_t h[kMaxBins];
    for (int b = threadIdx.x; b <= L; b += kGT) h[b] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * slice;
    for (int64_t i = i0 + threadIdx.x; i < i0 + slice && i < n; i += kGT) atomicAdd(&h[bin_of(leaves, i, L)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b <= L; b += kGT) hist[b * bin_step + blockIdx.x * slice_step] = h[b];
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

// Places of one slice's slots.  FROM: 0 the slice is everything; 1 hist holds the slices' counts
// [slice][bin]; 2 hist holds the slots of earlier slices [bin][slice], total the bins' sums.
template <int FROM>
__global__ __launch_bounds__(kGT) void group_place_kernel(const int32_t* leaves, int64_t n, int32_t L, int32_t run,
                                                          const int32_t* hist, const int32_t* total, int64_t* offsets,
                                                          int32_t* order) {
    __shared__ int32_t cnt[kGW][kMaxBins];
    __shared__ int32_t wave_sum[kGW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, bins = L + 1;
    const int64_t r0 = (int64_t)blockIdx.x * run * kGW + wave * run;
    int32_t bin[kRounds];  // of this lane's slots, -1 past the end
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const int64_t i = r0 + k * 64 + lane;
        bin[k] = k * 64 < run && i < n ? bin_of(leaves, i, L) : -1;
    }
    for (int w = 0; w < kGW; ++w)
        for (int b = tid; b < bins; b += kGT) cnt[w][b] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRounds; ++k)
        if (bin[k] >= 0) atomicAdd(&cnt[wave][bin[k]], 1);
    __syncthreads();
    // rows of smaller bins: each thread scans a run of bins
    const int per = (bins + kGT - 1) / kGT, b0 = tid * per, b1 = b0 + per < bins ? b0 + per : bins;
    auto bin_total = [&](int b, int32_t* before) {  // all slots of bin b, those of earlier slices
        int32_t t = 0;
        *before = 0;
        if constexpr (FROM == 0) {
            for (int w = 0; w < kGW; ++w) t += cnt[w][b];
        } else if constexpr (FROM == 1) {
#pragma unroll 16
            for (uint32_t s = 0; s < gridDim.x; ++s) {
                const int32_t c = hist[(int64_t)s * bins + b];
                *before += s < blockIdx.x ? c : 0;
                t += c;
            }
        } else {
            t = total[b];
            *before = hist[(int64_t)b * gridDim.x + blockIdx.x];
        }
        return t;
    };
    int32_t sum = 0, before0 = 0;
    for (int b = b0; b < b1; ++b) sum += bin_total(b, &before0);
    const int32_t incl = wave_inclusive_sum(sum);
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    int32_t at = incl - sum;
    for (int w = 0; w < wave; ++w) at += wave_sum[w];
    for (int b = b0; b < b1; ++b) {
        if (blockIdx.x == 0) offsets[b] = at;  // bin L starts where the last leaf ends
        int32_t before = before0;
        const int32_t t = per == 1 ? sum : bin_total(b, &before);
        int32_t base = at + before;
        for (int w = 0; w < kGW; ++w) {
            const int32_t c = cnt[w][b];
            cnt[w][b] = base;
            base += c;
        }
        at += t;
    }
    __syncthreads();
    const int bits = 32 - __builtin_clz(bins);
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        if (k * 64 >= run) break;
        const int b = bin[k];
        uint64_t same = __ballot(b >= 0);
        for (int u = 0; u < bits; ++u) {
            const uint64_t m = __ballot((b >> u) & 1);
            same &= (b >> u) & 1 ? m : ~m;
        }
        const int rank = __popcll(same & lanemask_lt());
        if (b >= 0) {
            order[cnt[wave][b] + rank] = (int32_t)(r0 + k * 64 + lane);
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
            if (rank == 0) cnt[wave][b] += __popcll(same);
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// Slots of a wave's run: an even share of one slice; two rounds while that keeps the slices few.
int32_t run_of(int64_t n) {
    if (n <= kOneSlice) return n < 1 ? 64 : (int32_t)((n + kGW * 64 - 1) / (kGW * 64) * 64);
    return n <= (1 << 18) ? 128 : kRounds * 64;
}
int64_t slices_of(int64_t n) { return (n + kGW * run_of(n) - 1) / (kGW * run_of(n)); }

}  // namespace

size_t group_rows_workspace_bytes(int64_t n, int32_t L) {
    const int64_t s = slices_of(n);
    return s > 1 ? (size_t)(s + 1) * (L + 1) * sizeof(int32_t) : 0;
}

hipError_t launch_group_rows(const int32_t* leaves, int64_t n, int32_t L, int64_t* offsets, int32_t* order, void* ws,
                             hipStream_t stream) {
    const int64_t s = slices_of(n), bins = L + 1;
    const int32_t run = run_of(n);
    const dim3 grid((uint32_t)(s < 1 ? 1 : s)), block(kGT);
    if (s <= 1) {
        hipLaunchKernelGGL(group_place_kernel<0>, grid, block, 0, stream, leaves, n, L, run, nullptr, nullptr, offsets,
                           order);
        return hipGetLastError();
    }
    int32_t* total = static_cast<int32_t*>(ws);
    int32_t* hist = total + bins;
    if (s * bins <= kDirect) {
        hipLaunchKernelGGL(group_hist_kernel, grid, block, 0, stream, leaves, n, L, run * kGW, (int64_t)1, bins, hist);
        hipLaunchKernelGGL(group_place_kernel<1>, grid, block, 0, stream, leaves, n, L, run, hist, nullptr, offsets,
                           order);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(group_hist_kernel, grid, block, 0, stream, leaves, n, L, run * kGW, s, (int64_t)1, hist);
    hipLaunchKernelGGL(group_scan_kernel, dim3((uint32_t)(bins + 3) / 4), dim3(256), 0, stream, hist, s, (int32_t)bins,
                       total);
    hipLaunchKernelGGL(group_place_kernel<2>, grid, block, 0, stream, leaves, n, L, run, hist, total, offsets, order);
    return hipGetLastError();
}

}  // namespace ah
