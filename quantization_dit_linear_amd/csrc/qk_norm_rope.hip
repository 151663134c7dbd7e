// qk_norm_rope.hip -- RMS norm of every query and key head with the rotary
// embedding in the same pass.
//
//   n_i = x_i / sqrt(mean_j x_j^2 + eps) * w_i          (over one head)
//   (n_u, n_v) -> (n_u cos t - n_v sin t, n_u sin t + n_v cos t)
// with the pairs and angles of rope.hip: 64-bit fractions of a turn, a token's
// cosines and sines made once into LDS for all its heads.
//
// Memory bound: each head is read once, kept in registers between the sum of
// squares and the turn, and written once, 16 bytes a lane.  G neighbouring lanes
// share a head, so its sum is log2 G lane exchanges.
#include <hip/hip_runtime.h>

#include "mx_codec.h"
#include "oq_internal.h"
#include "rope_turn.h"

namespace oq {
namespace {

constexpr int kPairs = 1024;  // LDS table: pairs of the tokens that a workgroup takes

template <class T>
__device__ __forceinline__ void load_weight(const void *w, int dtype, int at, float *v) {
  constexpr int E = 16 / sizeof(T);
#pragma unroll
  for (int e = 0; e < E; e++)
    v[e] = !w ? 1.f
           : dtype == 1 ? __builtin_bit_cast(float, (uint32_t)((const uint16_t *)w)[at + e] << 16)
                        : ((const float *)w)[at + e];
}

// the sum over the G lanes of a head
template <int G>
__device__ __forceinline__ float head_sum(float v) {
  auto dpp = [](float x, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x),
                                                                 decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});   // lane ^ 1
  v += dpp(v, std::integral_constant<int, 0x4E>{});   // lane ^ 2
  v += dpp(v, std::integral_constant<int, 0x141>{});  // the other four of 8
  if constexpr (G > 8) v += dpp(v, std::integral_constant<int, 0x140>{});  // the other eight of 16
  if constexpr (G > 16) v += __shfl_xor(v, 16);
  if constexpr (G > 32) v += __shfl_xor(v, 32);
  return v;
}

// blockIdx.x: a group of tokens; blockIdx.y: a slice of `hs` heads, the keys'
// behind the queries'.  Lane c of a head's G takes items c, c + G: E elements of
// the head, 16 bytes (interleaved pairs), or elements u and v of E pairs
// (half-split); the items behind the turned ones are only normed.
template <class T, bool HALF, int G, int NI>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(QkNormRopeArgs a, int tok_group, int hs) {
  __shared__ __attribute__((aligned(16))) f32x2 table[kPairs + 8];
  constexpr int E = 16 / sizeof(T), R = 256 / G;  // heads a pass
  const int tid = threadIdx.x, half = a.turned / 2, lane = tid % G;
  const int h0 = blockIdx.y * hs, heads = a.side[0].heads + a.side[1].heads;
  const int nh = heads - h0 < hs ? heads - h0 : hs;
  const int turned_items = HALF ? half / E : (a.turned + E - 1) / E;
  const int per = HALF ? turned_items + (a.head_dim - a.turned) / E : a.head_dim / E;
  const float inv_d = 1.0f / (float)a.head_dim;
  const int dh = R % nh, dt = R / nh;

  float wu[2][NI][E], wv[2][NI][HALF ? E : 1];
  int at[NI];
#pragma unroll
  for (int i = 0; i < NI; i++) {
    const int c = lane + G * i;
    at[i] = c >= per ? -1 : !HALF || c < turned_items ? E * c : a.turned + E * (c - turned_items);
    if (at[i] < 0) continue;
#pragma unroll
    for (int s = 0; s < 2; s++) {
      load_weight<T>(a.side[s].weight, a.param_dtype, at[i], wu[s][i]);
      if constexpr (HALF)
        if (c < turned_items) load_weight<T>(a.side[s].weight, a.param_dtype, at[i] + half, wv[s][i]);
    }
  }

  for (int64_t t0 = (int64_t)blockIdx.x * tok_group; t0 < a.tokens;
       t0 += (int64_t)gridDim.x * tok_group) {
    const int nt = a.tokens - t0 < tok_group ? (int)(a.tokens - t0) : tok_group;
    __syncthreads();  // the table of the group before is read
    for (int i = tid; i < nt * half; i += 256) {
      const int t = i / half, j = i - t * half;
      const uint64_t f = (uint64_t)(int64_t)a.pos[(t0 + t) * a.axes + a.axis[j]] * a.freq[j];
      table[i] = cos_sin((uint32_t)((f + 0x80000000ull) >> 32));
    }
    __syncthreads();

    int h = tid / G, t = h / nh;
    h -= t * nh;
    while (t < nt) {
      const int s = h0 + h >= a.side[0].heads;
      const QkNormRopeArgs::Side &sd = a.side[s];
      const int64_t hh = h0 + h - (s ? a.side[0].heads : 0);
      const T *px = (const T *)sd.x + (t0 + t) * sd.x_token + hh * sd.x_head;
      T *py = (T *)sd.y + (t0 + t) * sd.y_token + hh * sd.y_head;
      float u[NI][E], v[NI][HALF ? E : 1];
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NI; i++) {
        if (at[i] < 0) continue;
        load16(px + at[i], u[i]);
        if constexpr (HALF)
          if (lane + G * i < turned_items) load16(px + at[i] + half, v[i]);
      }
      auto squares = [&](float unit) {
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < NI; i++) {
          if (at[i] < 0) continue;
#pragma unroll
          for (int e = 0; e < E; e++) {
            const float x = u[i][e] * unit;
            q = fmaf(x, x, q);
          }
          if constexpr (HALF)
            if (lane + G * i < turned_items)
#pragma unroll
              for (int e = 0; e < E; e++) {
                const float x = v[i][e] * unit;
                q = fmaf(x, x, q);
              }
        }
        return head_sum<G>(q);
      };
      ss = squares(1.f);
      const float ms = fmaf(ss, inv_d, a.eps);
      float rs = rsqrtf(ms), back = 1.f;
      if (__any(!(ms < __builtin_huge_valf()))) {
        // a mean overflowed: once more at 2^-72, where the squares of 512 values
        // below 2^128 sum to 2^121 at most.  The factor's 2^-72 is applied behind
        // the product, exactly.  (A head with a NaN or an infinity stays one.)
        const float m2 = fmaf(squares(0x1p-72f), inv_d, a.eps * 0x1p-144f);
        if (!(ms < __builtin_huge_valf())) rs = rsqrtf(m2), back = 0x1p-72f;
      }
#pragma unroll
      for (int i = 0; i < NI; i++) {
        const int c = lane + G * i;
        if (at[i] < 0) continue;
#pragma unroll
        for (int e = 0; e < E; e++) u[i][e] = u[i][e] * rs * back * (s ? wu[1][i][e] : wu[0][i][e]);
        if (c < turned_items) {
          const f32x2 *z = table + t * half + (HALF ? E : E / 2) * c;
          if constexpr (HALF) {
#pragma unroll
            for (int e = 0; e < E; e++) {
              const float x = u[i][e], y = v[i][e] * rs * back * (s ? wv[1][i][e] : wv[0][i][e]);
              u[i][e] = x * z[e][0] - y * z[e][1];
              v[i][e] = x * z[e][1] + y * z[e][0];
            }
            store16_nt(py + at[i] + half, v[i]);
          } else {
            const int left = half - E / 2 * c;  // the last item may hold elements behind the turned ones
#pragma unroll
            for (int e = 0; e < E / 2; e++) {
              if (e >= left) break;
              const float x = u[i][2 * e], y = u[i][2 * e + 1];
              u[i][2 * e] = x * z[e][0] - y * z[e][1];
              u[i][2 * e + 1] = x * z[e][1] + y * z[e][0];
            }
          }
        }
        store16_nt(py + at[i], u[i]);
      }
      h += dh, t += dt;
      if (h >= nh) h -= nh, t++;
    }
  }
}

template <class T, bool HALF>
void launch(const QkNormRopeArgs &a, dim3 grid, int group, int hs, int per) {
  const dim3 block(256);
#define OQ_CASE(G, NI) hipLaunchKernelGGL((qk_norm_rope_kernel<T, HALF, G, NI>), grid, block, 0, a.stream, a, group, hs)
  if (per <= 8) OQ_CASE(8, 1);
  else if (per <= 16) OQ_CASE(16, 1);
  else if (per <= 32) OQ_CASE(32, 1);
  else if (per <= 64) OQ_CASE(64, 1);
  else if constexpr (sizeof(T) == 4) OQ_CASE(64, 2);  // fp32 heads of more than 256
#undef OQ_CASE
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkNormRopeArgs &a) {
  // tokens a workgroup and slices of the heads as in launch_rope
  const int half = a.turned / 2, unit = a.dtype == 1 ? 8 : 4, most = half > 0 ? kPairs / half : 64;
  const int per = a.half ? half / unit + (a.head_dim - a.turned) / unit : a.head_dim / unit;
  const int64_t heads = (int64_t)a.side[0].heads + a.side[1].heads;
  const int64_t items = 1024 / (heads * per);
  int group = half > 0 ? 256 / half : 1;
  if (group < items) group = (int)items;
  if (group > most) group = most;
  if (group < 1 || a.tokens < 1024 * (int64_t)group) group = 1;
  const int64_t gx = (a.tokens + group - 1) / group;
  int64_t hs = heads;
  auto slices = [&] { return (heads + hs - 1) / hs; };
  while (gx * slices() < 1024 && hs * per > 256) hs = (hs + 1) / 2;
  if (slices() > 65535) hs = (heads + 65534) / 65535;
  const dim3 grid((unsigned)(gx < (1 << 20) ? gx : 1 << 20), (unsigned)slices());
  if (a.dtype == 0) {
    if (a.half) launch<float, true>(a, grid, group, (int)hs, per);
    else launch<float, false>(a, grid, group, (int)hs, per);
  } else {
    if (a.half) launch<uint16_t, true>(a, grid, group, (int)hs, per);
    else launch<uint16_t, false>(a, grid, group, (int)hs, per);
  }
  return hipGetLastError();
}

}  // namespace oq
