// rope.hip -- rotary embedding with one to four axes.
//
// The first R = sum of the axes' sizes elements of a head are R/2 pairs; pair
// i of axis a turns by the angle  t = p_a theta^(-2i / size_a):
//   (u, v) -> (u cos t - v sin t, u sin t + v cos t).
// Angles are counted in turns as 64-bit fractions: the host gives F =
// theta^(-2i/size) / 2 pi in units of 2^-64, and p F modulo 2^64 is the turn's
// fraction, exact to 2^-64 |p| at any position -- no reduction of a large
// floating-point angle.
#include <hip/hip_runtime.h>

#include "mx_codec.h"
#include "oq_internal.h"

namespace oq {
namespace {

// cos and sin of pair j at position p
__device__ __forceinline__ f32x2 turn(const RopeArgs &a, int64_t tok, int j) {
  const int64_t p = a.pos[tok * a.axes + a.axis[j]];
  const uint64_t f = (uint64_t)p * a.freq[j];
  // nearest multiple of 2^-32 turn, as a signed fraction in [-1/2, 1/2]
  const int32_t q = (int32_t)(uint32_t)((f + 0x80000000ull) >> 32);
  float s, c;
  sincospif((float)q * 0x1p-31f, &s, &c);
  return f32x2{c, a.inverse ? -s : s};
}

// One thread: 8 consecutive elements of a head (interleaved pairs), or the 8
// elements u and 8 elements v of pairs 8c .. 8c+7 (half-split).
template <class T, bool HALF>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
  const int per = HALF ? (a.turned / 16) + (a.head_dim - a.turned) / 8 : a.head_dim / 8;
  const int64_t n = a.tokens * a.heads * per;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < n; t += (int64_t)gridDim.x * 256) {
    const int c = (int)(t % per);
    const int64_t th = t / per, head = th % a.heads, tok = th / a.heads;
    const T *x = (const T *)a.x + tok * a.x_token + head * a.x_head;
    T *y = (T *)a.y + tok * a.y_token + head * a.y_head;
    float u[8];
    if (HALF && c < a.turned / 16) {
      const int half = a.turned / 2;
      float v[8];
      load8(x + 8 * c, u);
      load8(x + half + 8 * c, v);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const f32x2 z = turn(a, tok, 8 * c + k);
        const float p = u[k] * z[0] - v[k] * z[1], q = u[k] * z[1] + v[k] * z[0];
        u[k] = p, v[k] = q;
      }
      store8(y + 8 * c, u);
      store8(y + half + 8 * c, v);
    } else {
      const int at = HALF ? a.turned + 8 * (c - a.turned / 16) : 8 * c;
      load8(x + at, u);
      if (!HALF)
#pragma unroll
        for (int k = 0; k < 4; k++)
          if (at + 2 * k < a.turned) {
            const f32x2 z = turn(a, tok, at / 2 + k);
            const float p = u[2 * k] * z[0] - u[2 * k + 1] * z[1];
            const float q = u[2 * k] * z[1] + u[2 * k + 1] * z[0];
            u[2 * k] = p, u[2 * k + 1] = q;
          }
      store8(y + at, u);
    }
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a) {
  const int per = a.half ? (a.turned / 16) + (a.head_dim - a.turned) / 8 : a.head_dim / 8;
  const int64_t n = a.tokens * a.heads * per, g = (n + 255) / 256;
  const dim3 grid((unsigned)(g < 65536 ? g : 65536)), block(256);
#define OQ_CASE(DT, T, H)        \
  if (a.dtype == DT && a.half == H) \
    hipLaunchKernelGGL((rope_kernel<T, H>), grid, block, 0, a.stream, a);
  OQ_CASE(0, float, false) OQ_CASE(0, float, true)
  OQ_CASE(1, uint16_t, false) OQ_CASE(1, uint16_t, true)
#undef OQ_CASE
  return hipGetLastError();
}

}  // namespace oq
