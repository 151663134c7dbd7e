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

#ifndef KV_D
#define KV_D 2
#endif
constexpr int kWaves = 4;

template <int NB>
struct RowsShape {
  static constexpr int HD = 32 * NB;
  // tokens a step: 64 where their LDS rows leave room for two workgroups a CU
  static constexpr int TOK = kv_rows_step(HD), TS = TOK / 32;
  // LDS row of a token's values: 64 bytes past a multiple of 256, so that four
  // tokens' pieces fall into different banks
  static constexpr int ROWB = 2 * HD + (NB % 2 == 0 ? 64 : 0);
  static constexpr int WAVE_BYTES = TOK * ROWB;
};

// what one step needs from memory, as loaded
template <int NB>
struct Raw {
  static constexpr int W = NB % 4 == 0 ? 4 : NB % 2 == 0 ? 2 : 1;  // dwords of keys a load
  static constexpr int TS = RowsShape<NB>::TS, NL = NB / W, NV = (TS * NB + 1) / 2;
  uint32_t k[2 * TS][NL][W];
  uint32_t ks[2 * TS][NL];
  u32x4 v[NV];
  uint32_t vs[NV];
  uint64_t missing;  // tokens whose page is not there
};

template <int NB, int QT, bool F32>
__global__ __launch_bounds__(256, 2) void kv_rows_kernel(KvLaunch p) {
  using Shape = RowsShape<NB>;
  using T = typename std::conditional<F32, float, uint16_t>::type;
  constexpr int HD = Shape::HD, ROWB = Shape::ROWB, NQ = F32 ? 3 : 1;
  constexpr int W = Raw<NB>::W, NL = Raw<NB>::NL, NV = Raw<NB>::NV, TS = Shape::TS, TOK = Shape::TOK;
  __shared__ __attribute__((aligned(16))) char lds[kWaves * Shape::WAVE_BYTES];
  const KvAttentionArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, kg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // the same in all lanes, and so are the steps
  const int worker = (int)blockIdx.x * kWaves + wave;
  int share = 0, pos = 0, end = 1;
  if (p.workers) {
    share = share_of(p, end);
    pos = worker * share;
    end = pos + share < end ? pos + share : end;
  } else if (worker >= p.count) {
    return;
  }
  while (pos < end) {
  // the group, and this wave's steps of it
  KvTile t;
  int kh, g0 = 0, g1 = 1 << 30, slot = -1;
  if (p.workers) {
    const KvUnits u = find_units(p, pos);
    const int at = pos - u.before, g = at / u.units, skip = at - g * u.units;
    const int len = u.units - skip < end - pos ? u.units - skip : end - pos;
    t = u.t;
    kh = g / u.tiles;
    const int tile = g - kh * u.tiles;
    t.row0 = tile * p.rows;
    g1 = u.first + skip + len - p.extra;
    g0 = skip > p.extra ? u.first + skip - p.extra : u.first;
    if (len < u.units) slot = 2 * worker + (skip == 0);
    if (skip == 0 && lane == 0)
      p.parts[(int64_t)(u.tiles_before + tile) * a.cache.heads + kh] =
          int2{slot, (pos + u.units - 1) / share - worker + 1};
    pos += len;
  } else {
    t = find_tile(p, worker);
    kh = blockIdx.y;
    pos = end;
    if (t.b < 0) return;
  }
  // the rows of this lane's columns, their tokens and operands; columns behind
  // the last row repeat it and see nothing
  int lo[QT], hi[QT];
  bf16x8 qf[QT][NL * W][NQ];
#pragma unroll
  for (int x = 0; x < QT; x++) {
    const int r = t.row0 + 16 * x + col;
    uint32_t i, h;
    p.share.split((uint32_t)(r < t.rows ? r : t.rows - 1), i, h);
    seen(a, t, (int)i, lo[x], hi[x]);
    if (r >= t.rows) lo[x] = hi[x] = 0;
    const T *q = (const T *)a.q + (t.start + (int64_t)i) * a.q_token + ((int64_t)kh * p.share.d + h) * a.q_head;
    float v[NL * W][8];
#pragma unroll
    for (int s = 0; s < NL * W; s++)  // step s = (load, dword): as the keys below
      load8(q + 8 * ((4 * (s / W) + kg) * W + s % W), v[s]);
#pragma unroll
    for (int s = 0; s < NL * W; s++) {
      if (a.scale < 0.f)
#pragma unroll
        for (int k = 0; k < 8; k++) v[s][k] = -v[s][k];
      split8<NQ>(v[s], qf[x][s]);
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

  // the steps that any row of the tile sees, of those that are this workgroup's
  const int s0 = any_lo / TOK > g0 ? any_lo / TOK : g0;
  const int s1 = any_hi <= any_lo ? s0 : (any_hi + TOK - 1) / TOK < g1 ? (any_hi + TOK - 1) / TOK : g1;
  const int step0 = s0, step1 = s1;

  char *rows = lds + wave * Shape::WAVE_BYTES;
  // D steps are in flight.  Loads come back in order and a step's follow from its
  // page numbers, so these are requested 2 D steps ahead: waiting for them then
  // waits for no more than what is used next.  All loads are unconditional, so that
  // their number is known; behind the part's end they repeat its last token.
  constexpr int D = F32 || NB > 4 ? 1 : KV_D;
  const int last_tok = (TOK * step1 < any_hi ? TOK * step1 : any_hi) - 1;
  auto token = [&](int step) {
    const int tok = TOK * step + (lane & (TOK - 1));
    return tok < last_tok ? tok : last_tok;
  };
  // (without a table any word will do; the sequence's number stands for it)
  const int32_t *table = a.table ? a.table + (int64_t)t.b * a.table_pages : a.lengths + t.b;
  const uint32_t mask = a.table ? ~0u : 0u;
  auto entry = [&](int step) { return table[p.page.div((uint32_t)token(step)) & mask]; };
  auto load = [&](int step, int page, Raw<NB> &raw) {
    uint32_t pg, off;
    p.page.split((uint32_t)token(step), pg, off);
    page = a.table ? page : t.b;
    const bool there = (uint32_t)page < (uint64_t)a.cache.pages;
    raw.missing = __ballot(!there);
    const int64_t row = ((int64_t)(there ? page : 0) * a.cache.heads + kh) * a.cache.page + off;
    const int rl = (int)row, rh = (int)(row >> 32);
    auto from = [&](int src) { return (int64_t)__shfl(rh, src) << 32 | (uint32_t)__shfl(rl, src); };
#pragma unroll
    for (int i = 0; i < 2 * TS; i++) {
      const int64_t at = from(16 * i + col);
#pragma unroll
      for (int j = 0; j < NL; j++) {
        // the lane's keys: elements 8 ((4 load + kg) W + dword) and the seven behind
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
        raw.ks[i][j] = a.cache.k_scales[at * NB + w / 4];
      }
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int x = lane + 64 * i, tok = x / NB < TOK ? x / NB : TOK - 1, blk = x % NB;
      const int64_t at = from(tok);
      raw.v[i] = *(const u32x4 *)(a.cache.v_codes + at * (HD / 2) + 16 * blk);
      raw.vs[i] = a.cache.v_scales[at * NB + blk];
    }
  };

  auto consume = [&](int step, Raw<NB> &cur) {
    // what is rare, out of the way: scales of NaN, pages that are not there, tokens
    // outside of what the tile sees.  Values that no row may meet become zeros (of
    // blocks of NaN below, what they make of the rows that see them).
    bool odd = false;
#pragma unroll
    for (int i = 0; i < NV; i++) odd |= kv_nan(cur.vs[i]);
#pragma unroll
    for (int i = 0; i < 2 * TS; i++)
#pragma unroll
      for (int j = 0; j < NL; j++) odd |= kv_nan(cur.ks[i][j]);
    uint64_t nan[NV] = {};
    bool any_nan = false;
    if (__any(odd) || cur.missing || TOK * step < any_lo || TOK * step + TOK > any_hi) {
#pragma unroll
      for (int i = 0; i < NV; i++) {
        const int x = lane + 64 * i, tok = x / NB, at = TOK * step + tok;
        const bool in = tok < TOK && at >= any_lo && at < any_hi && !(cur.missing >> (tok & 63) & 1);
        nan[i] = __ballot(in && kv_nan(cur.vs[i]));
        any_nan |= nan[i] != 0;
        if (!in || kv_nan(cur.vs[i])) cur.v[i] = u32x4{0, 0, 0, 0}, cur.vs[i] = 127;
      }
#pragma unroll
      for (int i = 0; i < 2 * TS; i++)
#pragma unroll
        for (int j = 0; j < NL; j++)
          if (kv_nan(cur.ks[i][j]) || (cur.missing >> (16 * i + col) & 1)) cur.ks[i][j] = 255;
    }
    // values into the wave's LDS rows
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int x = lane + 64 * i, tok = x / NB, blk = x % NB;
      if (TOK * NB % 64 == 0 || tok < TOK)
#pragma unroll
        for (int c = 0; c < 4; c++)
          *(bf16x8 *)(rows + tok * ROWB + 64 * blk + 16 * (c ^ (tok & 3))) = fp4x8(cur.v[i][c], kv_scale(cur.vs[i]));
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();

    f32x4 s[QT][2 * TS];
#pragma unroll
    for (int i = 0; i < 2 * TS; i++) {
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
    const bool edge = TOK * step < all_lo || TOK * step + TOK > all_hi;
    bf16x8 pf[QT][TS][NQ];
#pragma unroll
    for (int x = 0; x < QT; x++) {
      float v[8 * TS];
#pragma unroll
      for (int e = 0; e < 8 * TS; e++) v[e] = s[x][e >> 2][e & 3];
      if (edge) {
#pragma unroll
        for (int e = 0; e < 8 * TS; e++) {
          const int tok = TOK * step + 16 * (e >> 2) + 4 * kg + (e & 3);
          if (tok < lo[x] || tok >= hi[x]) v[e] = -kInf;
        }
      }
      float top = v[0];
#pragma unroll
      for (int e = 1; e < 8 * TS; e++) top = fmaxf(top, v[e]);
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
      for (int e = 0; e < 8 * TS; e++) {
        v[e] = __builtin_amdgcn_exp2f(fmaf(v[e], p.log2_scale, -base));
        l[x] += v[e];
      }
#pragma unroll
      for (int h = 0; h < TS; h++) split8<NQ>(v + 8 * h, pf[x][h]);
    }
    // transposed reads: lanes 4j .. 4j+3 of 16 name token j's 16 elements
    const int j = col >> 2, c = col & 3;
    const char *vb = rows + (4 * kg + j) * ROWB + 8 * (c & 1);
#pragma unroll
    for (int d = 0; d < 2 * NB; d++) {
#pragma unroll
      for (int h = 0; h < TS; h++) {
        const char *at = vb + 32 * h * ROWB + 64 * (d >> 1) + 16 * ((2 * (d & 1) + (c >> 1)) ^ j);
        const i16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)at);
        const i16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(at + 16 * ROWB));
        const bf16x8 vt = __builtin_bit_cast(bf16x8, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
        for (int x = 0; x < QT; x++)
#pragma unroll
          for (int n = NQ - 1; n >= 0; n--)
            o[x][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pf[x][h][n], o[x][d], 0, 0, 0);
      }
    }
    if (any_nan) {
      // blocks of NaN among the values: NaN for the rows that see their tokens
#pragma unroll
      for (int i = 0; i < NV; i++) {
        for (uint64_t left = nan[i]; left; left &= left - 1) {
          const int x = __builtin_ctzll(left) + 64 * i, tok = TOK * step + x / NB, blk = x % NB;
#pragma unroll
          for (int y = 0; y < QT; y++)
#pragma unroll
            for (int d = 0; d < 2 * NB; d++)
              if (d >> 1 == blk && tok >= lo[y] && tok < hi[y]) o[y][d] += __builtin_nanf("");
        }
      }
    }
  };

  if (step0 < step1) {
    Raw<NB> ring[D];
    int page[D];
#pragma unroll
    for (int u = 0; u < D; u++) page[u] = entry(step0 + u);
#pragma unroll
    for (int u = 0; u < D; u++) {
      const int now = page[u];
      page[u] = entry(step0 + u + D);
      load(step0 + u, now, ring[u]);
      __builtin_amdgcn_sched_barrier(0);  // the order of the loads is what the waits go by
    }
    for (int step = step0;;) {
#pragma unroll
      for (int u = 0; u < D; u++) {
        consume(step, ring[u]);
        const int now = page[u];
        page[u] = entry(step + 2 * D);
        load(step + D, now, ring[u]);
        __builtin_amdgcn_sched_barrier(0);
        step++;
        if (step >= step1) goto done;
      }
    }
  done:;
  }

#pragma unroll
  for (int x = 0; x < QT; x++) {
    const int r = t.row0 + 16 * x + col;
    const float sum = sum_over_16s(l[x]);
    if (r < t.rows) {
      uint32_t i, h;
      p.share.split((uint32_t)r, i, h);
      const int64_t tok = t.start + (int64_t)i, head = (int64_t)kh * p.share.d + h;
      if (slot < 0) {
        T *out = (T *)a.out + tok * a.out_token + head * a.out_head;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int d = 0; d < 2 * NB; d++) store4(out + 16 * d + 4 * kg, sum == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : o[x][d] * inv);
        if (a.lse && kg == 0) a.lse[tok * a.q_heads + head] = lse_of(m[x], sum);
      } else {
        const int64_t at = (int64_t)slot * p.rows + 16 * x + col;
        if (kg == 0) p.part_ml[at] = f32x2{m[x], sum};
        if (sum != 0.f)
#pragma unroll
          for (int d = 0; d < 2 * NB; d++) *(f32x4 *)(p.part + at * HD + 16 * d + 4 * kg) = o[x][d];
      }
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

hipError_t launch_kv_rows(const KvLaunch &p) {
  const dim3 grid((unsigned)((p.workers ? p.workers : p.count) + kWaves - 1) / kWaves,
                  p.workers ? 1u : (unsigned)p.a.cache.heads);
  switch (p.a.cache.head_dim / 32) {
#define OQ_CASE(NB) \
  case NB: launch<NB>(p, grid); break;
    OQ_CASE(1) OQ_CASE(2) OQ_CASE(3) OQ_CASE(4) OQ_CASE(5) OQ_CASE(6) OQ_CASE(7) OQ_CASE(8)
#undef OQ_CASE
  }
  return hipGetLastError();
}

}  // namespace oq
