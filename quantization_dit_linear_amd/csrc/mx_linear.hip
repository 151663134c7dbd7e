// mx_linear.hip -- the linear on microscaled (MX) codes, gfx950 matrix cores.
//
//   y[m][n] = bf16( sum_b 2^(sa_mb + sw_nb - 254) sum_{k in block b} a_mk w_nk )
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies elements of either type and
// applies the two blocks' powers of two itself.  Lane (r = lane % 16, g =
// lane / 16) supplies row r.  4-bit elements: k = 32 g + [0, 32), one
// 16-byte word.  8-bit elements: k = 16 g + [0, 16) and 64 + 16 g + [0, 16).
// In both cases the lane's scale byte is that of k block g (k = 32 g ..).
#include <hip/hip_runtime.h>

#include "mx_codec.h"
#include "oq_internal.h"

namespace oq {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// One row's operand for k0 .. k0 + 127: zero codes and scales past K or the last row.
template <int FMT>
__device__ __forceinline__ void load_operand(const uint8_t *codes, const uint8_t *scales,
                                             int64_t row, bool in, int k0, int K, int g, i32x8 &v,
                                             int &s) {
  u32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
  s = 0;
  if (in) {
    if constexpr (FMT == 0) {
      if (k0 + 32 * g < K) lo = *(const u32x4 *)(codes + row * (K / 2) + k0 / 2 + 16 * g);
    } else {
      const uint8_t *p = codes + row * K + k0 + 16 * g;
      if (k0 + 16 * g < K) lo = *(const u32x4 *)p;
      if (k0 + 64 + 16 * g < K) hi = *(const u32x4 *)(p + 64);
    }
    if (k0 + 32 * g < K) s = scales[row * (K / 32) + k0 / 32 + g];
  }
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = (int)lo[i], v[4 + i] = (int)hi[i];
}

// A wave computes 16 x 16 outputs, weights as the first operand so that a
// lane ends up with 4 consecutive columns of one output row.
template <int FA, int FW>
__global__ __launch_bounds__(256) void mx_linear_kernel(
    const uint8_t *__restrict__ A, const uint8_t *__restrict__ As, const uint8_t *__restrict__ W,
    const uint8_t *__restrict__ Ws, int M, int N, int K, uint16_t *__restrict__ Y) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int nbn = (N + 15) / 16;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  const int m0 = (int)(t / nbn) * 16, n0 = (int)(t % nbn) * 16;
  if (m0 >= M) return;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < K; k0 += 128) {
    i32x8 a, w;
    int sa, sw;
    load_operand<FA>(A, As, m0 + r, m0 + r < M, k0, K, g, a, sa);
    load_operand<FW>(W, Ws, n0 + r, n0 + r < N, k0, K, g, w, sw);
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, acc, FW ? 0 : 4, FA ? 0 : 4, 0, sw,
                                                           0, sa);
  }
  const int m = m0 + r;
  if (m >= M) return;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int n = n0 + 4 * g + i;
    if (n < N) Y[(int64_t)m * N + n] = __builtin_bit_cast(uint16_t, (__bf16)acc[i]);
  }
}

}  // namespace

hipError_t launch_mx_linear(const MxLinearArgs &a) {
  const int64_t waves = ((a.M + 15) / 16) * ((a.N + 15) / 16), grid = (waves + 3) / 4;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
#define OQ_CASE(FA, FW)                                                                        \
  if (a.a_format == FA && a.w_format == FW)                                                    \
    hipLaunchKernelGGL((mx_linear_kernel<FA, FW>), dim3((unsigned)grid), dim3(256), 0, a.stream, \
                       a.a_codes, a.a_scales, a.w_codes, a.w_scales, (int)a.M, (int)a.N, a.K, a.y);
  OQ_CASE(0, 0) OQ_CASE(0, 1) OQ_CASE(1, 0) OQ_CASE(1, 1)
#undef OQ_CASE
  return hipGetLastError();
}

}  // namespace oq
