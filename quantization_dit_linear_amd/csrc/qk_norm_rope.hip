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
// share a head, so its sum is log2 G lane exchanges.  The weights lie in LDS: held in
// registers they are a chain of loads at every workgroup's start and a choice between
// the two sides for every element.  Measured: 32760 tokens x (40 + 40) heads x 128 bf16
// 272 us (weights in registers 300 us; in a row of calls 265 us, 5.1 TB/s); 5003 tokens x
// (16 + 4) heads x 96 fp32, half-split, 17.4 us (25.7 us; traced alone 21 us, in a row of
// calls 16.7 us); one token 4.1 us (6.0 us).  Two passes' loads at
// once against one, three and four: 272, 277, 278, 307 us.
#include <hip/hip_runtime.h>

#include "mx_codec.h"
#include "oq_internal.h"
#include "rope_turn.h"

namespace oq {
namespace {

constexpr int kMaxHeadDim = 512;
constexpr int kPairs = 1024;  // LDS table: pairs of the tokens that a workgroup takes

__device__ __forceinline__ void widen(u32x4 r, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; e++) {
    v[2 * e] = __builtin_bit_cast(float, r[e] << 16);
    v[2 * e + 1] = __builtin_bit_cast(float, r[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(u32x4 r, float (&v)[4]) {
  const f32x4 f = __builtin_bit_cast(f32x4, r);
#pragma unroll
  for (int e = 0; e < 4; e++) v[e] = f[e];
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
  __shared__ __attribute__((aligned(16))) float weight[2][kMaxHeadDim];
  constexpr int E = 16 / sizeof(T), R = 256 / G, U = 2;  // heads a pass, passes loaded at once
  const int tid = threadIdx.x, half = a.turned / 2, lane = tid % G;
  const int h0 = blockIdx.y * hs, heads = a.side[0].heads + a.side[1].heads;
  const int nh = heads - h0 < hs ? heads - h0 : hs;
  const int turned_items = HALF ? half / E : (a.turned + E - 1) / E;
  const int per = HALF ? turned_items + (a.head_dim - a.turned) / E : a.head_dim / E;
  const float inv_d = 1.0f / (float)a.head_dim;
  const int dh = R % nh, dt = R / nh;

  int at[NI];
#pragma unroll
  for (int i = 0; i < NI; i++) {
    const int c = lane + G * i;
    at[i] = c >= per ? -1 : !HALF || c < turned_items ? E * c : a.turned + E * (c - turned_items);
  }
  for (int i = tid; i < 2 * a.head_dim; i += 256) {
    const int s = i >= a.head_dim, e = i - (s ? a.head_dim : 0);
    const void *const w = a.side[s].heads ? a.side[s].weight : nullptr;
    weight[s][e] = !w ? 1.f
                   : a.param_dtype == 1 ? __builtin_bit_cast(float, (uint32_t)((const uint16_t *)w)[e] << 16)
                                        : ((const float *)w)[e];
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
    // U heads at a time, all loads first; what is behind the last reads the first
    while (t < nt) {
      u32x4 ru[U][NI], rv[U][HALF ? NI : 1];
      int it[U], is[U];
      T *py[U];
#pragma unroll
      for (int k = 0; k < U; k++) {
        it[k] = t;
        const int tc = t < nt ? t : 0, hc = t < nt ? h0 + h : h0;
        const int s = is[k] = hc >= a.side[0].heads;
        const QkNormRopeArgs::Side &sd = a.side[s];
        const int64_t hh = hc - (s ? a.side[0].heads : 0);
        const T *px = (const T *)sd.x + (t0 + tc) * sd.x_token + hh * sd.x_head;
        py[k] = (T *)sd.y + (t0 + tc) * sd.y_token + hh * sd.y_head;
#pragma unroll
        for (int i = 0; i < NI; i++) {
          const T *src = px + (at[i] < 0 ? 0 : at[i]);
          ru[k][i] = *(const u32x4 *)src;
          if constexpr (HALF) rv[k][i] = *(const u32x4 *)(lane + G * i < turned_items ? src + half : src);
        }
        h += dh, t += dt;
        if (h >= nh) h -= nh, t++;
      }
#pragma unroll
      for (int k = 0; k < U; k++) {
        if (it[k] >= nt) break;
        const int s = is[k];
        float u[NI][E], v[NI][HALF ? E : 1];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NI; i++) {
          widen(ru[k][i], u[i]);
          if constexpr (HALF) widen(rv[k][i], v[i]);
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
        const bool rare = __any(!(ms < __builtin_huge_valf()));
        if (rare) {
          // a mean overflowed: once more at 2^-72, where the squares of 512 values
          // below 2^128 sum to 2^121 at most.  The factor's 2^-72 is applied behind
          // the product, exactly.  (A head with a NaN or an infinity stays one.)
          const float m2 = fmaf(squares(0x1p-72f), inv_d, a.eps * 0x1p-144f);
          if (!(ms < __builtin_huge_valf())) rs = rsqrtf(m2), back = 0x1p-72f;
        }
        const auto normed = [&](float (&x)[E], int at) {
#pragma unroll
          for (int e = 0; e < E; e++) x[e] *= rs;
          if (rare)
#pragma unroll
            for (int e = 0; e < E; e++) x[e] *= back;
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            const f32x4 w = *(const f32x4 *)(weight[s] + at + e);
#pragma unroll
            for (int j = 0; j < 4; j++) x[e + j] *= w[j];
          }
        };
#pragma unroll
        for (int i = 0; i < NI; i++) {
          const int c = lane + G * i;
          if (at[i] < 0) continue;
          normed(u[i], at[i]);
          if (c < turned_items) {
            const f32x2 *z = table + it[k] * half + (HALF ? E : E / 2) * c;
            if constexpr (HALF) {
              normed(v[i], at[i] + half);
#pragma unroll
              for (int e = 0; e < E; e++) {
                const float x = u[i][e], y = v[i][e];
                u[i][e] = x * z[e][0] - y * z[e][1];
                v[i][e] = x * z[e][1] + y * z[e][0];
              }
              store16_nt(py[k] + at[i] + half, v[i]);
            } else {
              const int left = half - E / 2 * c;  // the last item may hold elements behind the turned ones
#pragma unroll
              for (int e = 0; e < E / 2; e++) {
                const f32x2 r = e < left ? z[e] : f32x2{1.f, 0.f};
                const float x = u[i][2 * e], y = u[i][2 * e + 1];
                const float p = x * r[0] - y * r[1], q = x * r[1] + y * r[0];
                u[i][2 * e] = e < left ? p : x;
                u[i][2 * e + 1] = e < left ? q : y;
              }
            }
          }
          store16_nt(py[k] + at[i], u[i]);
        }
      }
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
