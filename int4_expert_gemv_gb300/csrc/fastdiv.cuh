// fastdiv.cuh -- division by a number that only the host knows beforehand.
#pragma once

#include <cstdint>

namespace moe {

// Division of 0 <= n < 2^31 by a divisor known on the host: with s = ceil(log2
// d) and m = floor(2^32 (2^s - d) / d) + 1, floor(n / d) = (hi(n m) + n) >> s
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994).
struct FastDiv {
    int d;
    uint32_t m;
    int s;
    FastDiv() = default;
    explicit FastDiv(int div) : d(div), s(0) {
        while (((int64_t)1 << s) < div) s++;
        m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - (uint64_t)div)) / (uint64_t)div + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int div(int n) const {
        return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> s);
    }
    __device__ __forceinline__ int ceil(int n) const {
        const int q = div(n);
        return q + (q * d != n);
    }
#endif
};

}  // namespace moe
