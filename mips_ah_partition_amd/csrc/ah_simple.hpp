// The plainest product: one workgroup of 256 threads has 64 rows x 64 columns, takes 16 elements of the sum at a
// time through LDS and adds in float32.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ah {

// q(row, t) and p(h, column, t): operands as float32 (zero outside); end(row, column, sums).
template <int NP, class Q, class P, class E>
__device__ __forceinline__ void simple_tile(int64_t red, Q q, P p, E end) {
    __shared__ float sq[16][65], sp[NP][16][65];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4][NP] = {};
    for (int64_t t0 = 0; t0 < red; t0 += 16) {
        for (int i = threadIdx.x; i < 64 * 16; i += 256) {
            const int t = i & 15, r = i >> 4;
            sq[t][r] = t0 + t < red ? q(r, t0 + t) : 0.0f;
            for (int h = 0; h < NP; ++h) sp[h][t][r] = t0 + t < red ? p(h, r, t0 + t) : 0.0f;
        }
        __syncthreads();
        for (int t = 0; t < 16; ++t)
            for (int r = 0; r < 4; ++r)
                for (int c = 0; c < 4; ++c)
                    for (int h = 0; h < NP; ++h) acc[r][c][h] += sq[t][ty * 4 + r] * sp[h][t][tx * 4 + c];
        __syncthreads();
    }
    for (int r = 0; r < 4; ++r)
        for (int c = 0; c < 4; ++c) end(ty * 4 + r, tx * 4 + c, acc[r][c]);
}

}  // namespace ah
