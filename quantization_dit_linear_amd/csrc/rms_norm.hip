// rms_norm.hip -- gated residual sum, RMS norm and modulation of a row, with
// the normalised row in the stream's own type or in microscaled codes.
//
//   h_i = r_i + g_i x_i
//   y_i = h_i / sqrt(mean_j h_j^2 + eps) * w_i (1 + a_i) + b_i
//
// The sum is written rounded to the stream's type; the norm runs over the
// unrounded fp32 sum, so y carries one rounding (and the codes none but
// their own).
//
// Memory bound: every row is read once, kept in registers between the sum
// of squares and the scaling, and written once.  64 to 512 threads take a row
// (by its length alone, so that a row's bits do not depend on the batch), a
// workgroup one row or a few short ones: workgroups that walk the rows with
// their parameters held in registers and the next row prefetched were 10%
// slower (32760 x 5120: 280 against 255 us), the parameters come from the L2.
// Stores are non-temporal (30000 x 512: 24 against 20 us).
//
// Measured: 32760 x 5120 bf16 230 us (5.8 TB/s; a large copy 5.3), with gate
// and modulation 249 us (5.4), that into e4m3 259 us (4.6), into e2m1 245 us
// (4.5); 9216 x 12288 184 us (4.9); fp32 4111 x 1536 22.4 us (4.5).  One row of
// 5120: 4.8 us, one wait for memory after another.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "mx_codec.h"
#include "oq_internal.h"

namespace oq {
namespace {

// 8 elements as loaded
template <class T>
struct Raw;
template <>
struct Raw<uint16_t> {
  u32x4 w;
  __device__ __forceinline__ void load(const uint16_t *p) { w = *(const u32x4 *)p; }
  __device__ __forceinline__ void get(float *v) const { unpack8(w, v); }
  __device__ __forceinline__ void fill(float f) {
    const uint32_t b = __builtin_bit_cast(uint32_t, f) >> 16;
    w = u32x4{b | b << 16, b | b << 16, b | b << 16, b | b << 16};
  }
};
template <>
struct Raw<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float *p) { a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4); }
  __device__ __forceinline__ void get(float *v) const {
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = a[i], v[4 + i] = b[i];
  }
  __device__ __forceinline__ void fill(float f) { a = b = f32x4{f, f, f, f}; }
};

__device__ __forceinline__ float wave_sum(float v) {
  auto dpp = [](float x, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x),
                                                                 decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});   // lane ^ 1
  v += dpp(v, std::integral_constant<int, 0x4E>{});   // lane ^ 2
  v += dpp(v, std::integral_constant<int, 0x141>{});  // the other four of 8
  v += dpp(v, std::integral_constant<int, 0x140>{});  // the other eight of 16
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// T: stream type, P: parameter type, TPR threads a row, NCH 8-element chunks
// a thread; MOD: with gate, scale or shift.
template <class T, class P, int TPR, int NCH, bool MOD>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256, 2) void rms_norm_kernel(RmsNormArgs a) {
  constexpr int TH = TPR > 256 ? TPR : 256;  // threads a workgroup
  constexpr int RPW = TH / TPR, WPR = TPR / 64, WAVES = TH / 64;  // rows a workgroup, waves a row
  // a bf16 weight is requested with the row (229 against 241 us at 32760 x
  // 5120); more parameters than that, where they are used (242 against 254 us):
  // waves in flight count more than the wait for the caches
  constexpr bool EARLY = sizeof(P) == 2 && !MOD;
  __shared__ float part[2][WAVES];
  const int tid = threadIdx.x, slot = tid / TPR, lt = tid % TPR, nch = a.d / 8;
  const float inv_d = 1.0f / (float)a.d;
  auto load_rest = [&](bool on, int c, int64_t mod, Raw<P> &w, Raw<P> &s, Raw<P> &b) {
    if (on && a.weight) w.load((const P *)a.weight + 8 * c);
    else w.fill(1.f);
    if constexpr (MOD) {
      if (on && a.scale) s.load((const P *)a.scale + mod + 8 * c);
      else s.fill(0.f);
      if (on && a.shift) b.load((const P *)a.shift + mod + 8 * c);
      else b.fill(0.f);
    }
  };

  int par = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * RPW; r0 < a.rows; r0 += (int64_t)gridDim.x * RPW) {
    const int64_t row = r0 + slot, mod = MOD ? row / a.rows_per_mod * a.mod_stride : 0;
    const bool in = row < a.rows;
    // everything the row needs is requested before any of it is used
    Raw<T> nx[NCH], nr[NCH];
    Raw<P> pw[NCH], pg[NCH], ps[NCH], pb[NCH];
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      const int c = lt + TPR * i;
      const bool on = in && c < nch;
      if (on) nx[i].load((const T *)a.x + row * a.d + 8 * c);
      if (on && a.residual) nr[i].load((const T *)a.residual + row * a.d + 8 * c);
      if constexpr (MOD) {
        if (on && a.gate) pg[i].load((const P *)a.gate + mod + 8 * c);
        else pg[i].fill(1.f);
      }
      if constexpr (EARLY) load_rest(on, c, mod, pw[i], ps[i], pb[i]);
    }
    float h[NCH][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      if (!in || lt + TPR * i >= nch) {
#pragma unroll
        for (int k = 0; k < 8; k++) h[i][k] = 0.f;
        continue;
      }
      nx[i].get(h[i]);
      if constexpr (MOD) {
        float g[8];
        pg[i].get(g);
#pragma unroll
        for (int k = 0; k < 8; k++) h[i][k] *= g[k];
      }
      if (a.residual) {
        float r[8];
        nr[i].get(r);
#pragma unroll
        for (int k = 0; k < 8; k++) h[i][k] += r[k];
      }
#pragma unroll
      for (int k = 0; k < 8; k++) ss = fmaf(h[i][k], h[i][k], ss);
    }

    // the mean of squares and eps; of a row times `unit`, with eps brought there too
    auto mean = [&](float sum, float unit) { return fmaf(sum, inv_d, a.eps * unit * unit); };
    // the row's total; `other`: any row of the workgroup whose mean is not finite
    auto total = [&](float v, bool &other) {
      v = wave_sum(v);
      if constexpr (WPR > 1) {
        if ((tid & 63) == 0) part[par][tid >> 6] = v;
        __syncthreads();
        float all[WAVES], t = 0.f;
        other = false;
#pragma unroll
        for (int w = 0; w < WAVES; w++) all[w] = part[par][w];
#pragma unroll
        for (int s = 0; s < RPW; s++) {
          float u = all[s * WPR];
#pragma unroll
          for (int w = 1; w < WPR; w++) u += all[s * WPR + w];
          other |= !(mean(u, 1.f) < __builtin_huge_valf());
          if (s == slot) t = u;
        }
        par ^= 1;
        return t;
      } else {
        other = !(mean(v, 1.f) < __builtin_huge_valf());
        return v;
      }
    };
    bool redo;
    ss = total(ss, redo);
    const float ms = mean(ss, 1.f);
    float rs = rsqrtf(ms), back = 1.f;
    if (redo) {
      // a mean overflowed: once more at 2^-72, where the squares of 16384
      // values below 2^128 sum to 2^126 at most, and those of a row whose sum
      // passed 2^128 to 2^-16 at least.  The factor's 2^-72 is applied behind
      // the product, exactly: 1 / rms itself may be subnormal.  (A row with a
      // NaN or an infinity stays one.)
      float s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NCH; i++)
#pragma unroll
        for (int k = 0; k < 8; k++) {
          const float t = h[i][k] * 0x1p-72f;
          s2 = fmaf(t, t, s2);
        }
      s2 = total(s2, redo);
      if (!(ms < __builtin_huge_valf())) rs = rsqrtf(mean(s2, 0x1p-72f)), back = 0x1p-72f;
    }
    if (!in) continue;
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      const int c = lt + TPR * i;
      if (c >= nch) continue;
      if (a.sum) store8_nt((T *)a.sum + row * a.d + 8 * c, h[i]);
      float y[8], w[8];
      if constexpr (!EARLY) load_rest(true, c, mod, pw[i], ps[i], pb[i]);
      pw[i].get(w);
#pragma unroll
      for (int k = 0; k < 8; k++) y[k] = h[i][k] * rs * back;
      if constexpr (MOD) {
        float s[8], b[8];
        ps[i].get(s), pb[i].get(b);
#pragma unroll
        for (int k = 0; k < 8; k++) y[k] = fmaf(y[k], w[k] * (1.0f + s[k]), b[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; k++) y[k] *= w[k];
      }
      if (a.out == 0) store8_nt((T *)a.y + row * a.d + 8 * c, y);
      else if (a.out == 1) mx_store8<1>(y, row * nch + c, (uint8_t *)a.y, a.y_scales);
      else mx_store8<0>(y, row * nch + c, (uint8_t *)a.y, a.y_scales);
    }
  }
}

template <class T, class P, bool MOD>
hipError_t launch_d(const RmsNormArgs &a) {
  auto go = [&](auto kernel, int rows_per_wg, int threads = 256) {
    const int64_t wgs = (a.rows + rows_per_wg - 1) / rows_per_wg;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(wgs < (1 << 20) ? wgs : 1 << 20)), dim3(threads), 0, a.stream, a);
    return hipGetLastError();
  };
  const int d = a.d;
  if (d <= 512) return go(rms_norm_kernel<T, P, 64, 1, MOD>, 4);
  if (d <= 1024) return go(rms_norm_kernel<T, P, 64, 2, MOD>, 4);
  if (d <= 2048) return go(rms_norm_kernel<T, P, 64, 4, MOD>, 4);
  if (d <= 5 * 1024) return go(rms_norm_kernel<T, P, 128, 5, MOD>, 2);
  if (d <= 8 * 1024) return go(rms_norm_kernel<T, P, 256, 4, MOD>, 1);
  return go(rms_norm_kernel<T, P, 512, 4, MOD>, 1, 512);
}

template <class T, class P>
hipError_t launch_mod(const RmsNormArgs &a) {
  return a.gate || a.scale || a.shift ? launch_d<T, P, true>(a) : launch_d<T, P, false>(a);
}

}  // namespace

hipError_t launch_rms_norm(const RmsNormArgs &a) {
  if (a.dtype == 0)
    return a.param_dtype == 0 ? launch_mod<float, float>(a) : launch_mod<float, uint16_t>(a);
  return a.param_dtype == 0 ? launch_mod<uint16_t, float>(a) : launch_mod<uint16_t, uint16_t>(a);
}

}  // namespace oq
