// rtn4_group.hip -- INT4 weights with a scale (and zero point) for every group
// of coordinates, and the projection of few rows by them.
//
//   y[m][n] = bf16( sum_g s_ng sum_{k in g} x_mk (nibble_nk - z_ng) )
#include <hip/hip_runtime.h>

#include <type_traits>

#include "kv_cache.h"
#include "mx_codec.h"
#include "oq_internal.h"

namespace oq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

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

// Eight lanes a group: each holds every eighth 8-element piece of it, read twice (the
// second time from cache), one element a load.  Runs once for a weight, so no more was
// done: 30720 x 5120 in groups of 64, bf16 309 us, fp32 544 us (1.3 TB/s).
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

// A few rows read every weight once: bound by memory up to some 16 rows, beyond that
// by the products and what prepares them.  A workgroup makes 16 NT columns of y for 16
// MT rows of x, its waves share K, and LDS joins their sums in a fixed order: one
// launch, 160 workgroups even where N is 5120.  A step is 128 coordinates.
//
// A nibble becomes the bf16 16 + nibble by one shift and one mask-or for two (its
// four bits are the upper mantissa bits of 16..31), so the products are exact in the
// matrix unit; a second product by ones gives sum x, and at a group's end
//   total += scale (sum x (16 + nibble) + (-16 - zero) sum x)
// in fp32.  fp32 activations are three exact bf16 parts, the small ones added first.
//
// The loads follow the rows in memory: four lanes take 64 bytes of a weight row, as
// many as 32 coordinates need take a part of an activation row, one load brings 16
// rows' scales of four groups.  LDS of the wave's own turns them to the lanes that the
// products want.  Loaded straight to those lanes (each lane of a load in a row of its
// own) the same kernel is held by address processing: 2 x 30720 x 5120 with zeros in 45
// instead of 30 us, 16 rows of 30720 x 5120 in 45 instead of 24 us.
//
// Launches of a graph, groups of 128 in bf16 where not said otherwise: 1 x 5120 x 5120
// 6.4 us; 1 x 32768 x 16384 55.6 us (5.0 TB/s); 2 x 30720 x 5120, groups of 64 with zeros,
// 24 us; 29 fp32 rows x 13824 x 5120, groups of 32, 32.5 us, half of it vector instructions
// (the parts, the nibbles, the groups' ends); 64 rows x 30720 x 5120 59 us and 512 rows
// 421 us: 32 rows a tile, each of which converts the weights again.
//
// GK: the group where it is 32, 64 or 128 (its products are known then, and the first
// starts from zero: 34.8 against 38.5 us for the 29 rows, 7.1 against 7.6 for one), else
// 0.  XR: the rows of x that there can be in a tile, 4 or 16; 4 are repeated, which
// saves three of four loads.
template <int MT, int NT, int XR, int WAVES, int GK, bool F32>
__global__ __launch_bounds__(64 * WAVES) void rtn4_group_linear_kernel(Rtn4GroupArgs a, FastDiv per_group) {
  constexpr int NQ = F32 ? 3 : 1, ES = F32 ? 4 : 2, XV = ES / 2;  // XV: 16-byte parts of 8 activations
  constexpr int C = XR == 4 ? 16 : 4 * XV, R = 64 / C;            // a load of x: rows and parts of a row
  constexpr int XD = XR == 4 ? 4 / XV : 1;                        // and the products that it serves
  constexpr int XL = MT * XR / R;                                 // loads of XD products
  constexpr int XS = MT > 1 && F32 ? 2 : 4 / XD;                  // such sets of loads in flight
  // No branch for a step's tail within it, so that one group's end overlaps the next
  // one's products: 2 x 30720 x 5120 in groups of 64 22.3 against 24.3 us.  Groups of 32
  // (29.3 to 35.7 us) and tiles of 64 columns lose their registers to it.
  constexpr bool STRAIGHT = GK == 64 && NT <= 2;
  constexpr int kSwap = 64 * (NT + XL), kPart = 4 * MT * (16 * NT + 4), kRegion = kSwap > kPart ? kSwap : kPart;
  __shared__ u32x4 region[WAVES][kRegion];
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, kg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16 * NT, m0 = (int64_t)blockIdx.y * 16 * MT;
  const int K = a.K, group = a.group, groups = K / group;
  const int steps = (K + 127) / 128, per = (steps + WAVES - 1) / WAVES;
  const int s0 = wave * per, s1 = s0 + per < steps ? s0 + per : steps;
  const int end = s1 * 128 < K ? s1 * 128 : K;

  // a uniform base and a lane's offset; rows behind the last are the last again:
  // their results are not used
  const char *const w_base = (const char *)a.q4 + n0 * (K / 2), *const x_base = (const char *)a.x + m0 * K * ES;
  const bool s32 = a.scale_dtype == 0, symmetric = !a.zeros;
  uint32_t row[NT], x_off[XL];
#pragma unroll
  for (int t = 0; t < NT; t++) {
    const uint32_t last = (uint32_t)(a.N - 1 - n0 < 16 * NT ? a.N - 1 - n0 : 16 * NT - 1), r = 16 * t + lane / 4;
    row[t] = r < last ? r : last;
  }
#pragma unroll
  for (int j = 0; j < XL; j++) {
    const uint32_t last = (uint32_t)(a.M - 1 - m0 < 16 * MT ? a.M - 1 - m0 : 16 * MT - 1), r = R * j + lane / C;
    x_off[j] = (r < last ? r : last) * K * ES;
  }
  u32x4 *const w_swap = region[wave], *const x_swap = w_swap + 64 * NT;
  // places of 16 bytes, turned so that eight lanes that read meet no bank twice
  const int w_put = lane / 4 * 4 + ((lane ^ lane / 16) & 3), w_get = col * 4 + ((kg ^ col / 4) & 3);
  const auto x_place = [&](int r, int c) {
    return r * C + (XR == 4 ? c ^ 4 * r : F32 ? c ^ 2 * (r / 2 & 3) : c ^ (r / 4 & 3));
  };
  const int x_row = XR == 4 ? col & 3 : col;
  // Between one lane's writes and another's reads of the wave's LDS, both ways: the
  // hardware keeps a wave's LDS operations in their order, this keeps the compiler to it
  // (no instruction of its own).
  const auto turn = [] {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };

  u32x4 w[NT], x[XS][XL];
  uint32_t sr[2][NT], zr[2][NT];  // scales and zeros of 16 rows x 4 groups, and of the next 4
  // what lies behind K is read inside the row and not used
  const auto load_w = [&](int s) {
    const int last = (K - s * 128) / 2 - 16;
    const uint32_t at = GK == 128 || 16 * (lane & 3) < last ? 16 * (lane & 3) : last;
#pragma unroll
    for (int t = 0; t < NT; t++) w[t] = *(const u32x4 *)(w_base + s * 64 + (row[t] * (K / 2) + at));
  };
  const auto load_x = [&](int s, int d) {  // d: of 4 / XD, then of the next step
    s += d / (4 / XD), d %= 4 / XD;
    s = s < s1 ? s : s1 - 1;
    const int c = (s * 128 + 32 * XD * d) * ES + lane % C * 16, last = K * ES - 16;
    const uint32_t at = GK == 128 || c < last ? c : last;
#pragma unroll
    for (int j = 0; j < XL; j++) x[d % XS][j] = *(const u32x4 *)(x_base + (x_off[j] + at));
  };
  const auto load_scales = [&](int quad, uint32_t (&sv)[NT], uint32_t (&zv)[NT]) {
    const int g = 4 * quad + (lane & 3);
    const int64_t at = n0 * groups + (g < groups ? g : groups - 1);
#pragma unroll
    for (int t = 0; t < NT; t++) {
      if (s32) sv[t] = ((const uint32_t *)a.scales)[at + row[t] * groups];
      else sv[t] = ((const uint16_t *)a.scales)[at + row[t] * groups];
      if (symmetric) zv[t] = 0;
      else if (s32) zv[t] = ((const uint32_t *)a.zeros)[at + row[t] * groups];
      else zv[t] = ((const uint16_t *)a.zeros)[at + row[t] * groups];
    }
  };

  f32x4 total[NT][MT], acc[NT][MT], sum[MT];
#pragma unroll
  for (int i = 0; i < MT; i++) {
    sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < NT; t++) total[t][i] = acc[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  bf16x8 ones;
#pragma unroll
  for (int e = 0; e < 8; e++) ones[e] = (__bf16)1.f;

  // in registers, so that and and or are one instruction (which takes no two literals)
  uint32_t mask = 0x00780078u, sixteen = 0x41804180u;
  asm("" : "+s"(mask), "+v"(sixteen));

  int g = 0, left = 0;  // the group, and the coordinates that it still holds
  float scale[NT], off[NT];
  const int up = s32 ? 0 : 16;
  const auto pick = [&] {
    const int from = 4 * (4 * col + (g & 3));
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const uint32_t sv = __builtin_amdgcn_ds_bpermute(from, sr[0][t]);
      scale[t] = __builtin_bit_cast(float, sv << up);
      off[t] = -24.f;
      if (!symmetric) {
        const uint32_t zv = __builtin_amdgcn_ds_bpermute(from, zr[0][t]);
        off[t] = -16.f - __builtin_bit_cast(float, zv << up);
      }
    }
  };
  if (s0 < s1) {
    g = per_group.div(4 * s0), left = (g + 1) * group - s0 * 128;
    load_scales(g / 4, sr[0], zr[0]);
    load_w(s0);
#pragma unroll
    for (int d = 0; d < XS; d++) load_x(s0, d);
    load_scales(g / 4 + 1, sr[1], zr[1]);
    pick();
  }
  for (int s = s0; s < s1; s++) {
    u32x4 q[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) w_swap[64 * t + w_put] = w[t];
    turn();
#pragma unroll
    for (int t = 0; t < NT; t++) q[t] = w_swap[64 * t + w_get];
    load_w(s + 1 < s1 ? s + 1 : s);
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const auto s02 = __builtin_amdgcn_permlane32_swap(q[t][0], q[t][2], false, false);
      const auto s13 = __builtin_amdgcn_permlane32_swap(q[t][1], q[t][3], false, false);
      const auto s01 = __builtin_amdgcn_permlane16_swap(s02[0], s13[0], false, false);
      const auto s23 = __builtin_amdgcn_permlane16_swap(s02[1], s13[1], false, false);
      q[t] = u32x4{s01[0], s01[1], s23[0], s23[1]};
    }
#pragma unroll
    for (int d = 0; d < 4; d++) {
      const int c = s * 128 + 32 * d;
      if (!STRAIGHT && GK != 128 && c >= end) break;
      if (d % XD == 0) {
        turn();
#pragma unroll
        for (int j = 0; j < XL; j++) x_swap[x_place(R * j + lane / C, lane % C)] = x[d / XD % XS][j];
        turn();
        load_x(s, d / XD + XS);
      }
      const bool fresh = GK && 32 * d % (GK ? GK : 1) == 0;
      const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
      // the activations in the order of the weights' pairs: coordinates j and j + 4
      bf16x8 xf[MT][NQ];
#pragma unroll
      for (int i = 0; i < MT; i++) {
        u32x4 v[XV];
#pragma unroll
        for (int e = 0; e < XV; e++) v[e] = x_swap[16 * C * i + x_place(x_row, 4 * XV * (d % XD) + XV * kg + e)];
        if constexpr (F32) {
#pragma unroll
          for (int e = 0; e < 8; e++) {
            float r = __builtin_bit_cast(f32x4, v[e & 1])[e / 2];
#pragma unroll
            for (int k = 0; k < NQ; k++) {
              xf[i][k][e] = (__bf16)r;
              if (k + 1 < NQ) r -= (float)xf[i][k][e];
            }
          }
        } else {
          const u32x4 p = {__builtin_amdgcn_perm(v[0][2], v[0][0], 0x05040100u), __builtin_amdgcn_perm(v[0][2], v[0][0], 0x07060302u),
                           __builtin_amdgcn_perm(v[0][3], v[0][1], 0x05040100u), __builtin_amdgcn_perm(v[0][3], v[0][1], 0x07060302u)};
          xf[i][0] = __builtin_bit_cast(bf16x8, p);
        }
#pragma unroll
        for (int k = NQ - 1; k >= 0; k--)  // small parts first
          sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i][k], ones, fresh && k == NQ - 1 ? zero : sum[i], 0, 0, 0);
      }
#pragma unroll
      for (int t = 0; t < NT; t++) {
        const uint32_t v = q[t][d];
        const u32x4 p = {(v << 3 & mask) | sixteen, (v >> 1 & mask) | sixteen, (v >> 5 & mask) | sixteen, (v >> 9 & mask) | sixteen};
        const bf16x8 wf = __builtin_bit_cast(bf16x8, p);
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
          for (int k = NQ - 1; k >= 0; k--)
            acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i][k], wf, fresh && k == NQ - 1 ? zero : acc[t][i], 0, 0, 0);
      }
      if (GK && (32 * d + 32) % (GK ? GK : 1)) continue;
      left -= 32;
      if (GK || left == 0 || c + 32 == end) {  // the group's end, or the wave's
#pragma unroll
        for (int i = 0; i < MT; i++) {
#pragma unroll
          for (int t = 0; t < NT; t++) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const float with = fmaf(scale[t], fmaf(off[t], sum[i][e], acc[t][i][e]), total[t][i][e]);
              // STRAIGHT: a step's second group may lie behind K.  It is made of the row's
              // last values, over and over, whose sums may pass the fp32 range where no
              // group's do: the total without it, not with 0 times it.
              total[t][i][e] = !STRAIGHT || d == 1 || c < end ? with : total[t][i][e];
            }
            if (!GK) acc[t][i] = zero;
          }
          if (!GK) sum[i] = zero;
        }
        g++, left = group;
        if ((!STRAIGHT || d == 3) && g % 4 == 0) {
#pragma unroll
          for (int t = 0; t < NT; t++) sr[0][t] = sr[1][t], zr[0][t] = zr[1][t];
          load_scales(g / 4 + 1, sr[1], zr[1]);
        }
        pick();
      }
    }
  }

  // the waves' sums, in their order
  float *const part = (float *)region;
  const auto at = [](int w, int m, int n) { return 4 * kRegion * w + (16 * NT + 4) * m + n; };
#pragma unroll
  for (int i = 0; i < MT; i++)
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int e = 0; e < 4; e++) part[at(wave, 16 * i + 4 * kg + e, 16 * t + col)] = total[t][i][e];
  __syncthreads();
  const int rows_here = a.M - m0 < 16 * MT ? (int)(a.M - m0) : 16 * MT;
  for (int e = tid; e < rows_here * 16 * NT; e += 64 * WAVES) {
    const int m = e / (16 * NT), n = e % (16 * NT);
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; w++) y += part[at(w, m, n)];
    if (n0 + n < a.N) a.y[(m0 + m) * a.N + n0 + n] = __builtin_bit_cast(uint16_t, (__bf16)y);
  }
}

template <int MT, int NT, int XR, int WAVES = 8>
void launch_linear(const Rtn4GroupArgs &a) {
  const dim3 grid((unsigned)((a.N + 16 * NT - 1) / (16 * NT)), (unsigned)((a.M + 16 * MT - 1) / (16 * MT))), block(64 * WAVES);
  const FastDiv per_group((uint32_t)(a.group / 32));
#define OQ_CASE(GK)                                                                                                     \
  {                                                                                                                     \
    if (a.dtype == 0) hipLaunchKernelGGL((rtn4_group_linear_kernel<MT, NT, XR, WAVES, GK, true>), grid, block, 0, a.stream, a, per_group); \
    else hipLaunchKernelGGL((rtn4_group_linear_kernel<MT, NT, XR, WAVES, GK, false>), grid, block, 0, a.stream, a, per_group); \
  }
  if (a.group == 128) OQ_CASE(128)
  else if (a.group == 64) OQ_CASE(64)
  else if (a.group == 32) OQ_CASE(32)
  else OQ_CASE(0)
#undef OQ_CASE
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

hipError_t launch_rtn4_group_linear(const Rtn4GroupArgs &all) {
  // Four tiles of columns share what a tile of x costs, two make twice the workgroups:
  // four win from 128 of them on (64 rows of 5120 x 5120, 160: 13.2 against 17.2 us;
  // 29 x 13824, 216: 14.7 against 18.7 us; not yet at 128 itself: 40 rows of 4096 x 16384
  // 34.8 against 24.7 us), two below (32 rows of 5120 x 13824, 80: 21.8 against 30.4
  // us).  Up to 16 rows two win over one and four (5120 x 5120: 7.9
  // against 8.3 and 11.3 us; 2 x 30720 x 5120: 21.3 against 22.9 and 24.4 us).
  const bool wide = ((all.N + 63) / 64) * ((all.M + 31) / 32) >= 128;
  // Where even tiles of 16 columns are a workgroup a CU at most: these, with sixteen
  // waves up to 16 rows (1 x 1024 x 16384, groups of 64: 9.8 us, eight waves 14.4, two
  // tiles 17.6; of K 4096 4.7, 5.0 and 6.3 us; 40 rows, eight waves: 19.0 against 26.7).
  const bool few = ((all.N + 15) / 16) * ((all.M + 31) / 32) <= 256;
  constexpr int64_t kRows = 1 << 20;  // a launch: a grid has no more than 65535 tiles of rows
  for (int64_t m = 0; m < all.M; m += kRows) {
    Rtn4GroupArgs a = all;
    a.x = (const char *)all.x + m * all.K * (all.dtype == 0 ? 4 : 2);
    a.y = all.y + m * all.N;
    a.M = all.M - m < kRows ? all.M - m : kRows;
    if (few && all.M <= 4) launch_linear<1, 1, 4, 16>(a);
    else if (few && all.M <= 16) launch_linear<1, 1, 16, 16>(a);
    else if (few) launch_linear<2, 1, 16>(a);
    else if (all.M <= 4) launch_linear<1, 2, 4>(a);
    else if (all.M <= 16) launch_linear<1, 2, 16>(a);
    else if (wide) launch_linear<2, 4, 16>(a);
    else launch_linear<2, 2, 16>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace oq
