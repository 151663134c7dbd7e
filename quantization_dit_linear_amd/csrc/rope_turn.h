// rope_turn.h -- cosine and sine of a fraction of a turn, for the kernels that
// apply the rotary embedding.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_codec.h"

namespace oq {

// (cos, sin) of 2 pi q / 2^32.  The nearest quarter turn apart, |x| <= pi/4,
// where the Taylor polynomials to x^10 and x^9 are within 2e-9.
__device__ __forceinline__ f32x2 cos_sin(uint32_t q) {
  const uint32_t n = (q + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(q - (n << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float z = x * x;
  float s = 1.f / 362880.f, c = -1.f / 3628800.f;
  s = fmaf(s, z, -1.f / 5040.f);
  s = fmaf(s, z, 1.f / 120.f);
  s = fmaf(s, z, -1.f / 6.f);
  s = fmaf(s * z, x, x);
  c = fmaf(c, z, 1.f / 40320.f);
  c = fmaf(c, z, -1.f / 720.f);
  c = fmaf(c, z, 1.f / 24.f);
  c = fmaf(c, z, -0.5f);
  c = fmaf(c, z, 1.f);
  const float a = n & 1 ? -s : c, b = n & 1 ? c : s;
  return n & 2 ? f32x2{-a, -b} : f32x2{a, b};
}

}  // namespace oq
