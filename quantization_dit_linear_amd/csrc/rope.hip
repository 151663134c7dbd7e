// rope.hip -- rotary embedding with one to four axes.
//
// The first R = sum of the axes' sizes elements of a head are R/2 pairs; pair
// i of axis a turns by the angle  t = p_a theta^(-2i / size_a):
//   (u, v) -> (u cos t - v sin t, u sin t + v cos t).
// Angles are counted in turns as 64-bit fractions: the host gives F =
// theta^(-2i/size) / 2 pi in units of 2^-64, and p F modulo 2^64 is the turn's
// fraction at any int32 position -- no reduction of a large floating-point
// angle, and no error that grows with the position beyond F's own rounding.
//
// Memory bound: x read and y written once, 16 bytes a lane.  A token's cosines
// and sines serve all its heads, so a workgroup computes them once into LDS
// (for several tokens, so that every thread has a pair to work on) and then
// streams the heads.  Measured: 32760 tokens x 80 heads x 128 bf16, strided
// input, 257 us (5.2 TB/s; each thread computing its own: 443 us); half-split 251
// us; 40 heads of fp32 259 us; 24 heads of 64: 35 us (5.7 TB/s); two heads of
// 128: 12.7 us (2.6 TB/s, the table's arithmetic); one token 3.9 us.
#include <hip/hip_runtime.h>

#include "mx_codec.h"
#include "oq_internal.h"
#include "rope_turn.h"

namespace oq {
namespace {

constexpr int kPairs = 1024;  // LDS table: pairs of the tokens that a workgroup takes

// blockIdx.x: a group of tokens; blockIdx.y: a slice of `hs` heads.  One item:
// E consecutive elements of a head, 16 bytes (interleaved pairs), or elements
// u and v of pairs E c .. E c + E - 1 (half-split); the items behind them copy.
template <class T, bool HALF>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, int tok_group, int hs) {
  __shared__ __attribute__((aligned(16))) f32x2 table[kPairs + 8];
  constexpr int E = 16 / sizeof(T);
  const int tid = threadIdx.x, half = a.turned / 2;
  const int h0 = blockIdx.y * hs, nh = a.heads - h0 < hs ? a.heads - h0 : hs;

  // items (token, head, c), c fastest; a thread's next is 256 further on
  const int turned_items = HALF ? half / E : (a.turned + E - 1) / E;
  const int per = HALF ? turned_items + (a.head_dim - a.turned) / E : a.head_dim / E;
  const int dc = 256 % per, dh = 256 / per % nh, dt = 256 / per / nh;

  for (int64_t t0 = (int64_t)blockIdx.x * tok_group; t0 < a.tokens;
       t0 += (int64_t)gridDim.x * tok_group) {
    const int nt = a.tokens - t0 < tok_group ? (int)(a.tokens - t0) : tok_group;
    __syncthreads();  // the table of the group before is read
    for (int i = tid; i < nt * half; i += 256) {
      const int t = i / half, j = i - t * half;
      const uint64_t f = (uint64_t)(int64_t)a.pos[(t0 + t) * a.axes + a.axis[j]] * a.freq[j];
      f32x2 z = cos_sin((uint32_t)((f + 0x80000000ull) >> 32));
      if (a.inverse) z[1] = -z[1];
      table[i] = z;
    }
    __syncthreads();

    int c = tid % per, h = tid / per, t = h / nh;
    h -= t * nh;
    const T *xb = (const T *)a.x + t0 * a.x_token + (int64_t)h0 * a.x_head;
    T *yb = (T *)a.y + t0 * a.y_token + (int64_t)h0 * a.y_head;
    auto next = [&] {
      c += dc, h += dh, t += dt;
      if (c >= per) c -= per, h++;
      if (h >= nh) h -= nh, t++;
    };
    // four items at a time, all loads first
    constexpr int U = 4;
    while (t < nt) {
      float u[U][E], v[U][E];
      int it[U], ic[U];
      const T *px[U];
      T *py[U];
#pragma unroll
      for (int k = 0; k < U; k++) {
        it[k] = t, ic[k] = c;
        const int at = !HALF || c < turned_items ? E * c : a.turned + E * (c - turned_items);
        px[k] = xb + t * a.x_token + (int64_t)h * a.x_head + at;
        py[k] = yb + t * a.y_token + (int64_t)h * a.y_head + at;
        if (t < nt) {
          load16(px[k], u[k]);
          if (HALF && c < turned_items) load16(px[k] + half, v[k]);
        }
        next();
      }
#pragma unroll
      for (int k = 0; k < U; k++) {
        if (it[k] >= nt) break;
        if (ic[k] < turned_items) {
          const f32x2 *z = table + it[k] * half + (HALF ? E : E / 2) * ic[k];
          if constexpr (HALF) {
#pragma unroll
            for (int e = 0; e < E; e++) {
              const float p = u[k][e] * z[e][0] - v[k][e] * z[e][1];
              v[k][e] = u[k][e] * z[e][1] + v[k][e] * z[e][0];
              u[k][e] = p;
            }
            store16_nt(py[k] + half, v[k]);
          } else {
            // the last item may hold elements behind the turned ones
            const int left = half - E / 2 * ic[k];
#pragma unroll
            for (int e = 0; e < E / 2; e++) {
              const f32x2 w = e < left ? z[e] : f32x2{1.f, 0.f};
              const float p = u[k][2 * e] * w[0] - u[k][2 * e + 1] * w[1];
              const float q = u[k][2 * e] * w[1] + u[k][2 * e + 1] * w[0];
              u[k][2 * e] = e < left ? p : u[k][2 * e];
              u[k][2 * e + 1] = e < left ? q : u[k][2 * e + 1];
            }
          }
        }
        store16_nt(py[k], u[k]);
      }
    }
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a) {
  // as many tokens a workgroup as give its threads a pair and four items
  // each, if that leaves 1024 workgroups (four a CU); else one token, and a
  // slice of the heads where the tokens alone are still fewer than that
  const int half = a.turned / 2, per = a.head_dim / 8, most = half > 0 ? kPairs / half : 64;
  const int64_t items = 1024 / ((int64_t)a.heads * per);
  int group = half > 0 ? 256 / half : 1;
  if (group < items) group = (int)items;
  if (group > most) group = most;
  if (group < 1 || a.tokens < 1024 * (int64_t)group) group = 1;
  const int64_t gx = (a.tokens + group - 1) / group;
  int64_t hs = a.heads;
  auto slices = [&] { return (a.heads + hs - 1) / hs; };
  while (gx * slices() < 1024 && hs * per > 256) hs = (hs + 1) / 2;
  const dim3 grid((unsigned)(gx < (1 << 20) ? gx : 1 << 20), (unsigned)slices()), block(256);
#define OQ_CASE(DT, T, H)        \
  if (a.dtype == DT && a.half == H) \
    hipLaunchKernelGGL((rope_kernel<T, H>), grid, block, 0, a.stream, a, group, (int)hs);
  OQ_CASE(0, float, false) OQ_CASE(0, float, true)
  OQ_CASE(1, uint16_t, false) OQ_CASE(1, uint16_t, true)
#undef OQ_CASE
  return hipGetLastError();
}

}  // namespace oq
