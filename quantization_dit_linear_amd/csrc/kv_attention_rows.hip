// kv_attention_rows.hip -- attention of few rows (single new tokens, short
// chunks) over the 4-bit cache.
//
// A workgroup's four waves take the 32-token steps of its part by turns, each
// with its own running maximum and sums, and join at the end.  A tile is 16 rows
// (or 32): rows are the queries of a sequence times the query heads of one key
// head, so shared heads read the cache once.  Per step a wave computes
//   S^T = K Q^T   (16x16x32 matrix instructions: tokens by rows),
// whose result leaves each lane four tokens of its row a time, in the order in
// which the second product
//   O^T = V^T P^T
// can take them as its operand: the contraction's slots are tokens in any order,
// so the weights never cross lanes.  Keys go from memory to registers, where 16
// bytes of codes are the operand after the conversion.  Values are converted a
// block a lane, written to the wave's own LDS rows and read back transposed;
// 16-byte pieces are swizzled by the token so that neither side conflicts.
#include <hip/hip_runtime.h>

#include "kv_attention.h"

namespace oq {
namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

constexpr int kWaves = 4;

template <int NB>
struct RowsShape {
  static constexpr int HD = 32 * NB;
  // LDS row of a token's values: 64 bytes past a multiple of 256, so that four
  // tokens' pieces fall into different banks
  static constexpr int ROWB = 2 * HD + (NB % 2 == 0 ? 64 : 0);
  static constexpr int OSTRIDE = HD + 4;  // floats of a row's sum in the join
  static constexpr int WAVE_BYTES = 32 * ROWB > 16 * OSTRIDE * 4 ? 32 * ROWB : 16 * OSTRIDE * 4;
};

// what one step needs from memory, as loaded
template <int NB>
struct Raw {
  static constexpr int W = NB % 4 == 0 ? 4 : NB % 2 == 0 ? 2 : 1;  // dwords of keys a load
  static constexpr int NL = NB / W, NV = (NB + 1) / 2;
  uint32_t k[2][NL][W];
  uint32_t ks[2][NL];
  u32x4 v[NV];
  uint32_t vs[NV];
};

template <int NB, int QT, bool F32>
__global__ __launch_bounds__(256) void kv_rows_kernel(KvLaunch p) {
  using Shape = RowsShape<NB>;
  using T = typename std::conditional<F32, float, uint16_t>::type;
  constexpr int HD = Shape::HD, ROWB = Shape::ROWB, NQ = F32 ? 3 : 1;
  constexpr int W = Raw<NB>::W, NL = Raw<NB>::NL, NV = Raw<NB>::NV;
  __shared__ __attribute__((aligned(16))) char lds[kWaves * Shape::WAVE_BYTES];
  __shared__ f32x2 ml[kWaves][16 * QT];
  const KvAttentionArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, kg = lane >> 4;
  const int kh = blockIdx.y, split = blockIdx.z;
  const KvTile t = find_tile(p, blockIdx.x);
  if (t.b < 0) return;

  // the rows of this lane's columns: their tokens and operands
  int lo[QT], hi[QT];
  bf16x8 qf[QT][NL * W][NQ];
#pragma unroll
  for (int x = 0; x < QT; x++) {
    const int r = t.row0 + 16 * x + col;
    lo[x] = hi[x] = 0;
    float v[8] = {};
    const bool in = r < t.rows;
    uint32_t i = 0, h = 0;
    if (in) {
      p.share.split((uint32_t)r, i, h);
      seen(a, t, (int)i, lo[x], hi[x]);
    }
    const T *q = (const T *)a.q + (t.start + (int64_t)i) * a.q_token + ((int64_t)kh * p.share.d + h) * a.q_head;
#pragma unroll
    for (int s = 0; s < NL * W; s++) {
      // step s = (load, dword): the lane's keys are elements 8 ((4 load + kg) W + dword)
      const int e = 8 * ((4 * (s / W) + kg) * W + s % W);
      if (in) load8(q + e, v);
      if (a.scale < 0.f)
#pragma unroll
        for (int k = 0; k < 8; k++) v[k] = -v[k];
      split8<NQ>(v, qf[x][s]);
    }
  }
  // what the tile as a whole sees, and what every row of it sees
  uint32_t first, last, unused;
  const int end = t.row0 + 16 * QT < t.rows ? t.row0 + 16 * QT : t.rows;
  p.share.split((uint32_t)t.row0, first, unused);
  p.share.split((uint32_t)(end - 1), last, unused);
  int any_lo, any_hi, all_lo, all_hi;
  seen(a, t, (int)first, any_lo, all_hi);
  seen(a, t, (int)last, all_lo, any_hi);

  f32x4 o[QT][2 * NB];
  float m[QT], l[QT];
#pragma unroll
  for (int x = 0; x < QT; x++) {
    m[x] = -kInf, l[x] = 0.f;
#pragma unroll
    for (int d = 0; d < 2 * NB; d++) o[x][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int s0 = any_lo / 32, s1 = any_hi > any_lo ? (any_hi + 31) / 32 : s0;
  const int per = (s1 - s0 + p.splits - 1) / p.splits;
  const int step0 = s0 + split * per + wave;
  const int step1 = s0 + (split + 1) * per < s1 ? s0 + (split + 1) * per : s1;

  char *rows = lds + wave * Shape::WAVE_BYTES;
  auto row_of = [&](int step) {
    const int tok = 32 * step + (lane & 31);
    return cache_row(p, t.b, kh, tok < any_hi ? tok : any_hi - 1);
  };
  auto load = [&](int step, int64_t row, Raw<NB> &raw) {
    const int rl = (int)row, rh = (int)(row >> 32);
    auto from = [&](int src) { return (int64_t)__shfl(rh, src) << 32 | (uint32_t)__shfl(rl, src); };
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int64_t r = from(16 * i + col), at = r < 0 ? 0 : r;
#pragma unroll
      for (int j = 0; j < NL; j++) {
        const int w = (4 * j + kg) * W;
        const uint32_t *src = (const uint32_t *)(a.cache.k_codes + at * (HD / 2)) + w;
        if constexpr (W == 4) {
          const u32x4 c = *(const u32x4 *)src;
#pragma unroll
          for (int e = 0; e < 4; e++) raw.k[i][j][e] = c[e];
        } else if constexpr (W == 2) {
          const u32x2 c = *(const u32x2 *)src;
          raw.k[i][j][0] = c[0], raw.k[i][j][1] = c[1];
        } else {
          raw.k[i][j][0] = *src;
        }
        raw.ks[i][j] = r < 0 ? 255 : a.cache.k_scales[at * NB + w / 4];
      }
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int x = lane + 64 * i, tok = x / NB, blk = x % NB;
      raw.v[i] = u32x4{0, 0, 0, 0};
      raw.vs[i] = 0;
      const int64_t r = from(tok & 31);
      // tokens that no row sees are zeros: what lies there may be NaN
      if (tok < 32 && r >= 0 && 32 * step + tok >= any_lo && 32 * step + tok < any_hi) {
        raw.v[i] = *(const u32x4 *)(a.cache.v_codes + r * (HD / 2) + 16 * blk);
        raw.vs[i] = a.cache.v_scales[r * NB + blk];
      }
    }
  };

  Raw<NB> cur, next;
  int64_t row = -1;
  if (step0 < step1) {
    load(step0, row_of(step0), cur);
    if (step0 + kWaves < step1) row = row_of(step0 + kWaves);
  }
  for (int step = step0; step < step1; step += kWaves) {
    if (step + kWaves < step1) {
      load(step + kWaves, row, next);
      if (step + 2 * kWaves < step1) row = row_of(step + 2 * kWaves);
    }
    // values into the wave's LDS rows; blocks of NaN as zeros, put right below
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int x = lane + 64 * i, tok = x / NB, blk = x % NB;
      const bool bad = kv_nan(cur.vs[i]);
      nan |= bad;
      const float s = mx_scale(bad ? 127 : cur.vs[i]);
      if (tok < 32)
#pragma unroll
        for (int c = 0; c < 4; c++)
          *(bf16x8 *)(rows + tok * ROWB + 64 * blk + 16 * (c ^ (tok & 3))) = fp4x8(bad ? 0u : cur.v[i][c], s);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();

    f32x4 s[QT][2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
#pragma unroll
      for (int x = 0; x < QT; x++) s[x][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NL; j++) {
        const float sc = kv_scale(cur.ks[i][j]);
#pragma unroll
        for (int w = 0; w < W; w++) {
          const bf16x8 k = fp4x8(cur.k[i][j][w], sc);
#pragma unroll
          for (int x = 0; x < QT; x++)
#pragma unroll
            for (int n = NQ - 1; n >= 0; n--)  // small parts first
              s[x][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, qf[x][j * W + w][n], s[x][i], 0, 0, 0);
        }
      }
    }
    const bool edge = 32 * step < all_lo || 32 * step + 32 > all_hi;
    bf16x8 pf[QT][NQ];
#pragma unroll
    for (int x = 0; x < QT; x++) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; e++) v[e] = s[x][e >> 2][e & 3];
      if (edge) {
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int tok = 32 * step + 16 * (e >> 2) + 4 * kg + (e & 3);
          if (tok < lo[x] || tok >= hi[x]) v[e] = -kInf;
        }
      }
      float top = v[0];
#pragma unroll
      for (int e = 1; e < 8; e++) top = fmaxf(top, v[e]);
      top = fmaxf(m[x], max_over_16s(top) * p.log2_scale);
      // a row that sees nothing yet keeps -infinity; 0 stands for it here
      const float base = top == -kInf ? 0.f : top;
      if (__any(top > m[x])) {
        const float old = __builtin_amdgcn_exp2f(m[x] - base);
        l[x] *= old;
#pragma unroll
        for (int d = 0; d < 2 * NB; d++) o[x][d] *= old;
        m[x] = top;
      }
#pragma unroll
      for (int e = 0; e < 8; e++) {
        v[e] = __builtin_amdgcn_exp2f(fmaf(v[e], p.log2_scale, -base));
        l[x] += v[e];
      }
      split8<NQ>(v, pf[x]);
    }
    // transposed reads: lanes 4j .. 4j+3 of 16 name token j's 16 elements
    const int j = col >> 2, c = col & 3;
    const char *vb = rows + (4 * kg + j) * ROWB + 8 * (c & 1);
#pragma unroll
    for (int d = 0; d < 2 * NB; d++) {
      const char *at = vb + 64 * (d >> 1) + 16 * ((2 * (d & 1) + (c >> 1)) ^ j);
      const i16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)at);
      const i16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(at + 16 * ROWB));
      const bf16x8 vt = __builtin_bit_cast(bf16x8, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
      for (int x = 0; x < QT; x++)
#pragma unroll
        for (int n = NQ - 1; n >= 0; n--)
          o[x][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pf[x][n], o[x][d], 0, 0, 0);
    }
    if (__any(nan)) {
      // blocks of NaN among the values: NaN for the rows that see their tokens
#pragma unroll
      for (int i = 0; i < NV; i++) {
        for (uint64_t left = __ballot(kv_nan(cur.vs[i])); left; left &= left - 1) {
          const int x = __builtin_ctzll(left) + 64 * i, tok = 32 * step + x / NB, blk = x % NB;
#pragma unroll
          for (int y = 0; y < QT; y++)
#pragma unroll
            for (int d = 0; d < 2 * NB; d++)
              if (d >> 1 == blk && tok >= lo[y] && tok < hi[y]) o[y][d] += __builtin_nanf("");
        }
      }
    }
    cur = next;
  }

  // the waves' sums, in their order
#pragma unroll
  for (int x = 0; x < QT; x++) {
    l[x] = sum_over_16s(l[x]);
    if (kg == 0) ml[wave][16 * x + col] = f32x2{m[x], l[x]};
  }
#pragma unroll
  for (int x = 0; x < QT; x++) {
    if (x > 0) __syncthreads();
    float *os = (float *)rows;
#pragma unroll
    for (int d = 0; d < 2 * NB; d++) *(f32x4 *)(os + col * Shape::OSTRIDE + 16 * d + 4 * kg) = o[x][d];
    __syncthreads();
    for (int e = tid; e < 16 * (HD / 4); e += 256) {
      const int c = e / (HD / 4), d = 4 * (e % (HD / 4)), r = t.row0 + 16 * x + c;
      if (r >= t.rows) break;
      float top = ml[0][16 * x + c][0], sum = 0.f;
#pragma unroll
      for (int w = 1; w < kWaves; w++) top = fmaxf(top, ml[w][16 * x + c][0]);
      const float base = top == -kInf ? 0.f : top;
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; w++) {
        const float f = __builtin_amdgcn_exp2f(ml[w][16 * x + c][0] - base);
        sum += ml[w][16 * x + c][1] * f;
        v += *(const f32x4 *)(lds + w * Shape::WAVE_BYTES + (c * Shape::OSTRIDE + d) * 4) * f;
      }
      uint32_t i, h;
      p.share.split((uint32_t)r, i, h);
      const int64_t tok = t.start + (int64_t)i, head = (int64_t)kh * p.share.d + h;
      const int64_t row = tok * a.q_heads + head;
      if (p.splits == 1) {
        const float inv = 1.f / sum;
        if (sum == 0.f) v = f32x4{0.f, 0.f, 0.f, 0.f};
        else v *= inv;
        store4((T *)a.out + tok * a.out_token + head * a.out_head + d, v);
        if (a.lse && d == 0) a.lse[row] = lse_of(top, sum);
      } else {
        const int64_t at = split * a.q_tokens * a.q_heads + row;
        if (d == 0) p.part_ml[at] = f32x2{top, sum};
        if (sum != 0.f) *(f32x4 *)(p.part + at * HD + d) = v;
      }
    }
  }
}

template <int NB>
void launch(const KvLaunch &p, dim3 grid) {
  if (p.a.dtype == 0) hipLaunchKernelGGL((kv_rows_kernel<NB, 1, true>), grid, dim3(256), 0, p.a.stream, p);
  else if (p.rows == 16) hipLaunchKernelGGL((kv_rows_kernel<NB, 1, false>), grid, dim3(256), 0, p.a.stream, p);
  else hipLaunchKernelGGL((kv_rows_kernel<NB, 2, false>), grid, dim3(256), 0, p.a.stream, p);
}

}  // namespace

hipError_t launch_kv_rows(const KvLaunch &p, int64_t tiles) {
  const dim3 grid((unsigned)tiles, (unsigned)p.a.cache.heads, (unsigned)p.splits);
  switch (p.a.cache.head_dim / 32) {
#define OQ_CASE(NB) \
  case NB: launch<NB>(p, grid); break;
    OQ_CASE(1) OQ_CASE(2) OQ_CASE(3) OQ_CASE(4) OQ_CASE(5) OQ_CASE(6) OQ_CASE(7) OQ_CASE(8)
#undef OQ_CASE
  }
  return hipGetLastError();
}

}  // namespace oq
