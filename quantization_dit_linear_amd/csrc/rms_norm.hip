// rms_norm.hip -- gated residual sum, RMS norm and modulation of a row, with
// the normalised row in the stream's own type or in microscaled codes.
//
//   h_i = r_i + g_i x_i
//   y_i = h_i / sqrt(mean_j h_j^2 + eps) * w_i (1 + a_i) + b_i
//
// The sum is written rounded to the stream's type; the norm runs over the
// unrounded fp32 sum, so y carries one rounding (and the codes none but
// their own).
#include <hip/hip_runtime.h>

#include "mx_codec.h"
#include "oq_internal.h"

namespace oq {
namespace {

// T: stream type, P: parameter type; OUT: 0 = y in T, 1 = e4m3, 2 = e2m1.
// One workgroup of 256 a row, the row in registers.
template <class T, class P, int OUT, int NCH>
__global__ __launch_bounds__(256) void rms_norm_kernel(RmsNormArgs a) {
  __shared__ float part[4];
  const int tid = threadIdx.x, nch = a.d / 8;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
  const int64_t grp = row / a.rows_per_mod;
  const T *x = (const T *)a.x + row * a.d, *res = (const T *)a.residual;
  float h[NCH][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; i++) {
    const int c = tid + 256 * i;
    if (c < nch) {
      load8(x + 8 * c, h[i]);
      if (a.gate) {
        float g[8];
        load8((const P *)a.gate + grp * a.mod_stride + 8 * c, g);
#pragma unroll
        for (int k = 0; k < 8; k++) h[i][k] *= g[k];
      }
      if (res) {
        float r[8];
        load8(res + row * a.d + 8 * c, r);
#pragma unroll
        for (int k = 0; k < 8; k++) h[i][k] += r[k];
      }
#pragma unroll
      for (int k = 0; k < 8; k++) ss += h[i][k] * h[i][k];
    }
  }
  auto total = [&](float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if ((tid & 63) == 0) part[tid >> 6] = v;
    __syncthreads();
    return part[0] + part[1] + part[2] + part[3];
  };
  ss = total(ss);
  const float inv_d = 1.0f / (float)a.d;
  float r;
  if (ss < __builtin_huge_valf()) {
    r = rsqrtf(ss * inv_d + a.eps);
  } else {
    // the squares overflowed: once more at 2^-64 (a row with a NaN or an
    // infinity stays one)
    float s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; i++)
      if (tid + 256 * i < nch)
#pragma unroll
        for (int k = 0; k < 8; k++) {
          const float t = h[i][k] * 0x1p-64f;
          s2 += t * t;
        }
    r = rsqrtf(total(s2) * inv_d) * 0x1p-64f;
  }
#pragma unroll
  for (int i = 0; i < NCH; i++) {
    const int c = tid + 256 * i;
    if (c >= nch) continue;
    if (a.sum) store8((T *)a.sum + row * a.d + 8 * c, h[i]);
    float y[8], p[8];
#pragma unroll
    for (int k = 0; k < 8; k++) y[k] = h[i][k] * r;
    if (a.weight) {
      load8((const P *)a.weight + 8 * c, p);
#pragma unroll
      for (int k = 0; k < 8; k++) y[k] *= p[k];
    }
    if (a.scale) {
      load8((const P *)a.scale + grp * a.mod_stride + 8 * c, p);
#pragma unroll
      for (int k = 0; k < 8; k++) y[k] *= 1.0f + p[k];
    }
    if (a.shift) {
      load8((const P *)a.shift + grp * a.mod_stride + 8 * c, p);
#pragma unroll
      for (int k = 0; k < 8; k++) y[k] += p[k];
    }
    if constexpr (OUT == 0)
      store8((T *)a.y + row * a.d + 8 * c, y);
    else
      mx_store8<OUT == 1 ? 1 : 0>(y, row * nch + c, (uint8_t *)a.y, a.y_scales);
  }
  }
}

template <class T, class P, int OUT>
hipError_t launch_d(const RmsNormArgs &a) {
  const int need = (a.d / 8 + 255) / 256;
  const dim3 g((unsigned)(a.rows < 65536 ? a.rows : 65536)), b(256);
#define OQ_CASE(n) \
  if (need <= n) { \
    hipLaunchKernelGGL((rms_norm_kernel<T, P, OUT, n>), g, b, 0, a.stream, a); \
    return hipGetLastError(); \
  }
  OQ_CASE(1) OQ_CASE(2) OQ_CASE(4) OQ_CASE(8)
#undef OQ_CASE
  return hipErrorInvalidValue;
}

template <class T, class P>
hipError_t launch_out(const RmsNormArgs &a) {
  if (a.out == 0) return launch_d<T, P, 0>(a);
  if (a.out == 1) return launch_d<T, P, 1>(a);
  return launch_d<T, P, 2>(a);
}

}  // namespace

hipError_t launch_rms_norm(const RmsNormArgs &a) {
  if (a.dtype == 0)
    return a.param_dtype == 0 ? launch_out<float, float>(a) : launch_out<float, uint16_t>(a);
  return a.param_dtype == 0 ? launch_out<uint16_t, float>(a) : launch_out<uint16_t, uint16_t>(a);
}

}  // namespace oq
