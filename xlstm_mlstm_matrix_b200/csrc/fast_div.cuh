// Division by a number known on the host, as a product: n / d for 0 <= n < 2^31 and 1 <= d < 2^31.
#pragma once
#include <stdint.h>

namespace xlstm {

struct FastDiv {
    uint32_t mul, shift, d;
};
// shift = ceil(log2 d), mul = floor(2^32 (2^shift - d) / d) + 1: then n / d = (hi32(mul n) + n) >> shift, exactly.
inline FastDiv fast_div(uint32_t d) {
    FastDiv f{0, 0, d};
    while ((1ull << f.shift) < d) ++f.shift;
    f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
    return f;
}
#ifdef __CUDACC__
__device__ __forceinline__ int quotient(int n, const FastDiv &f) {
    return (int)((__umulhi(f.mul, (uint32_t)n) + (uint32_t)n) >> f.shift);
}
// n becomes n mod d; returns n / d
__device__ __forceinline__ int split(int &n, const FastDiv &f) {
    const int q = quotient(n, f);
    n -= q * (int)f.d;
    return q;
}
#endif

}  // namespace xlstm
