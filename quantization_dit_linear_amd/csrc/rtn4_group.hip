// rtn4_group.hip -- INT4 weights with a scale (and zero point) for every group
// of coordinates, and the projection of few rows by them.
//
//   y[m][n] = bf16( sum_g s_ng sum_{k in g} x_mk (nibble_nk - z_ng) )
#include <hip/hip_runtime.h>

#include "mx_codec.h"
#include "oq_internal.h"

namespace oq {
namespace {

__device__ __forceinline__ float load_in(const void *x, int dtype, int64_t i) {
  return dtype == 1 ? __builtin_bit_cast(float, (uint32_t)((const uint16_t *)x)[i] << 16) : ((const float *)x)[i];
}

__device__ __forceinline__ float bf16_round(float v) {
  return __builtin_bit_cast(float, (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v) << 16);
}

__device__ __forceinline__ void store_scale(void *p, int dtype, int64_t i, float v) {
  if (dtype == 1) ((uint16_t *)p)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
  else ((float *)p)[i] = v;
}

// Eight lanes a group: each holds every eighth 8-element piece of it.
__global__ __launch_bounds__(256) void rtn4_group_prepare_kernel(const void *__restrict__ W, int dtype,
                                                                 int64_t groups, int group,
                                                                 uint32_t *__restrict__ q4,
                                                                 void *__restrict__ scales,
                                                                 void *__restrict__ zeros, int scale_dtype) {
  const int j = threadIdx.x & 7, pieces = group / 8;
  for (int64_t g = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3); g < groups; g += (int64_t)gridDim.x * 32) {
    float lo = 0.f, hi = 0.f;
    for (int p = j; p < pieces; p += 8)
      for (int e = 0; e < 8; e++) {
        const float w = load_in(W, dtype, g * group + 8 * p + e);
        lo = fminf(lo, w), hi = fmaxf(hi, w);
      }
    for (int off = 4; off > 0; off >>= 1) lo = fminf(lo, __shfl_xor(lo, off, 8)), hi = fmaxf(hi, __shfl_xor(hi, off, 8));
    // the definition's fp32 operations: IEEE division, round half to even
    float scale = zeros ? __fdiv_rn(hi, 15.f) - __fdiv_rn(lo, 15.f) : __fdiv_rn(fmaxf(hi, -lo), 7.f);
    if (scale_dtype == 1) scale = bf16_round(scale);
    float zero = 8.f;
    if (zeros) zero = scale > 0.f ? fminf(fmaxf(__builtin_rintf(__fdiv_rn(-lo, scale)), 0.f), 15.f) : 0.f;
    if (j == 0) {
      store_scale(scales, scale_dtype, g, scale);
      if (zeros) store_scale(zeros, scale_dtype, g, zero);
    }
    for (int p = j; p < pieces; p += 8) {
      uint32_t word = 0;
      for (int e = 0; e < 8; e++) {
        const float w = load_in(W, dtype, g * group + 8 * p + e);
        const float q = scale > 0.f ? __builtin_rintf(__fdiv_rn(w, scale)) : 0.f;
        word |= (uint32_t)(int)fminf(fmaxf(q + zero, 0.f), 15.f) << (4 * e);
      }
      q4[g * pieces + p] = word;
    }
  }
}

// One wave an output row, 8 coordinates a lane and step; rows of x in turn.
__global__ __launch_bounds__(256) void rtn4_group_linear_kernel(Rtn4GroupArgs a) {
  const int lane = threadIdx.x & 63, words = a.K / 8, groups = a.K / a.group;
  const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (n >= a.N) return;
  for (int64_t m = 0; m < a.M; m++) {
    float sum = 0.f;
    for (int w = lane; w < words; w += 64) {
      const int64_t g = n * groups + 8 * w / a.group;
      const float z = a.zeros ? load_in(a.zeros, a.scale_dtype, g) : 8.f;
      const uint32_t q = ((const uint32_t *)a.q4)[n * words + w];
      float v[8], t = 0.f;
      if (a.dtype == 1) load8((const uint16_t *)a.x + m * a.K + 8 * w, v);
      else load8((const float *)a.x + m * a.K + 8 * w, v);
#pragma unroll
      for (int e = 0; e < 8; e++) t = fmaf(v[e], (float)(q >> (4 * e) & 15) - z, t);
      sum = fmaf(load_in(a.scales, a.scale_dtype, g), t, sum);
    }
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    if (lane == 0) a.y[m * a.N + n] = __builtin_bit_cast(uint16_t, (__bf16)sum);
  }
}

}  // namespace

hipError_t launch_rtn4_group_prepare(const void *W, int dtype, int64_t rows, int d, int group,
                                     uint8_t *q4, void *scales, void *zeros, int scale_dtype,
                                     hipStream_t stream) {
  const int64_t groups = rows * (d / group), want = (groups + 31) / 32;
  hipLaunchKernelGGL(rtn4_group_prepare_kernel, dim3((unsigned)(want < 16384 ? want : 16384)), dim3(256), 0,
                     stream, W, dtype, groups, group, (uint32_t *)q4, scales, zeros, scale_dtype);
  return hipGetLastError();
}

hipError_t launch_rtn4_group_linear(const Rtn4GroupArgs &a) {
  hipLaunchKernelGGL(rtn4_group_linear_kernel, dim3((unsigned)((a.N + 3) / 4)), dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

}  // namespace oq
