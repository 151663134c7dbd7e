// kv_cache.h -- where a token's rows lie in the 4-bit key/value cache.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace oq {

// x / d and x % d for 0 <= x < 2^31, d >= 1: with l = ceil(log2 d) the product
// by m = ceil(2^(31 + l) / d) exceeds x / d by less than x d / (d 2^(31 + l)) <=
// 1 / d, so its whole part is the quotient's.
struct FastDiv {
  uint32_t d, m, s;
  explicit FastDiv(uint32_t div) : d(div) {
    uint32_t l = 0;
    while (((uint64_t)1 << l) < div) l++;
    s = 31 + l;
    m = (uint32_t)((((uint64_t)1 << s) + div - 1) / div);
  }
  __host__ __device__ uint32_t div(uint32_t x) const { return (uint32_t)((uint64_t)x * m >> s); }
  __host__ __device__ void split(uint32_t x, uint32_t &q, uint32_t &r) const {
    q = div(x);
    r = x - q * d;
  }
};

}  // namespace oq
