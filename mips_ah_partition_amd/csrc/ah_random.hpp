// Dropout's random numbers: Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", 2011), a function of a key and a counter, so that a mask is computed wherever it is needed and
// never stored.  Key: the caller's seed.  Counter: (column / 8, row, step).  A call gives 128 bits, 16 for each
// of eight columns; an element stays where its bits are at least t = min(rint(65536 p), 65535), so it is dropped with
// the probability t / 2^16, and those that stay are multiplied by 2^16 / (2^16 - t): unbiased for the p that
// is used, which is off from the given one by 2^-17 at most (above 1 - 2^-17, where t = 2^16 would leave nothing and
// an infinite factor, by less than 2^-16).  16 bits and not 32: half the generator's work, of which each round is
// two 32 x 32 -> 64 bit products.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ah {

struct Dropout {
    uint32_t t;           // 0: everything stays
    float factor;
    uint32_t k0, k1;      // the seed's halves
    const int64_t* step;  // device, or NULL: 0
};

inline Dropout make_dropout(double p, uint64_t seed, const int64_t* step) {
    const double r = __builtin_rint(65536.0 * p);
    const uint32_t t = r < 65535.0 ? (uint32_t)r : 65535u;
    return Dropout{t, (float)(65536.0 / (65536.0 - t)), (uint32_t)seed, (uint32_t)(seed >> 32), step};
}

// 16-bit numbers of columns 8 c8 .. 8 c8 + 7 of a row: number j is the low (j even) or high half of word j / 2.
struct Philox {
    uint32_t w[4];
    __device__ __forceinline__ uint32_t at(int j) const { return j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu; }
};
__device__ __forceinline__ Philox philox(const Dropout& d, uint64_t step, uint32_t row, uint32_t c8) {
    uint32_t a = c8, b = row, c = (uint32_t)step, e = (uint32_t)(step >> 32), k0 = d.k0, k1 = d.k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = (uint64_t)a * 0xD2511F53u, q = (uint64_t)c * 0xCD9E8D57u;
        a = (uint32_t)(q >> 32) ^ b ^ k0;
        b = (uint32_t)q;
        c = (uint32_t)(p >> 32) ^ e ^ k1;
        e = (uint32_t)p;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return Philox{{a, b, c, e}};
}
__device__ __forceinline__ uint64_t step_of_call(const Dropout& d) { return d.step ? (uint64_t)*d.step : 0u; }

}  // namespace ah
