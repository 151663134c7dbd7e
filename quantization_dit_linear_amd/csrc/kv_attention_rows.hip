// kv_attention_rows.hip -- attention of few rows (single new tokens, short
// chunks) over the 4-bit cache.
//
// A wave (or a team of four, by turns) takes its even share of all groups' steps,
// with its own running maximum and sums, and leaves a part for the join.  A group is a
// tile of 16 rows and a key head: rows are the queries of a sequence times the query
// heads of that key head, so shared heads read the cache once.  Per step a wave computes
//   S^T = K Q^T   (16x16x32 matrix instructions: tokens by rows),
// whose result leaves each lane four tokens of its row a time, in the order in
// which the second product
//   O^T = V^T P^T
// can take them as its operand: the contraction's slots are tokens in any order,
// so the weights never cross lanes.  Keys go from memory to registers, where 16
// bytes of codes are the operand after the conversion.  Values are converted a
// block a lane, written to the wave's own LDS rows and read back transposed;
// 16-byte pieces are swizzled by the token so that neither side conflicts.
//
// Bound by the cache's bytes where sequences are many: 64 of up to 8192 tokens (32
// query, 8 key heads of 128, 295 MB) 54 us and 6 us for the join, 5.4 TB/s; by
// latency where they are few: one of 32760 tokens 17 and 7 us.  By the parts between
// both: 8 of 4096 tokens with 16 rows a key head 40 us, three steps a wave, of which each
// leaves a part of 8 KB.  fp32 heads of 128 (27 registers), 224 (68) and 256 (95) and bf16
// heads of 224 (10) and 256 (26) spill: the 64 sequences 80 us in fp32, with heads of 256
// 153 us in bf16 (twice the bytes) and 290 us in fp32.
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
  // tokens a step: 64 where their LDS rows leave room for two workgroups a CU
  static constexpr int TOK = kv_rows_step(HD), TS = TOK / 32;
  // LDS row of a token's values: 64 bytes past a multiple of 256, so that four
  // tokens' pieces fall into different banks
  static constexpr int ROWB = 2 * HD + (NB % 2 == 0 ? 64 : 0);
  static constexpr int OSTRIDE = HD + 4;  // floats of a row's sum where a team joins
  // a wave's LDS: its values; for a team's join its rows' sums, maxima and sums of weights
  static constexpr int JOIN_BYTES = 16 * OSTRIDE * 4 + 16 * 8;
  static constexpr int WAVE_BYTES = TOK * ROWB > JOIN_BYTES ? TOK * ROWB : JOIN_BYTES;
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

template <int NB, bool F32>
__global__ __launch_bounds__(256, 2) void kv_rows_kernel(KvLaunch p) {
  using Shape = RowsShape<NB>;
  using T = typename std::conditional<F32, float, uint16_t>::type;
  constexpr int HD = Shape::HD, ROWB = Shape::ROWB, NQ = F32 ? 3 : 1;
  constexpr int W = Raw<NB>::W, NL = Raw<NB>::NL, NV = Raw<NB>::NV, TS = Shape::TS, TOK = Shape::TOK;
  __shared__ __attribute__((aligned(16))) char lds[kWaves * Shape::WAVE_BYTES];
  const KvAttentionArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, kg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // the same in all lanes, and so are the steps
  const int worker = p.team ? (int)blockIdx.x : (int)blockIdx.x * kWaves + wave;
  int share = 0, pos = 0, end = 1;
  KvUnits u;
  if (p.workers) u = first_units(p, worker, share, pos, end);
  else if (worker >= p.count) return;
  for (bool again = false; pos < end; again = true) {
  // the group, and this wave's steps of it
  KvTile t;
  int kh, g0 = 0, g1 = 1 << 30, slot = -1;
  if (p.workers) {
    if (again) u = find_units(p, pos);
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
  t = uniform(t), kh = uniform(kh), g0 = uniform(g0), g1 = uniform(g1), slot = uniform(slot), pos = uniform(pos);
  // what the tile as a whole sees, and what every row of it sees
  int any_lo, any_hi, all_lo, all_hi;
  const int row1 = t.row0 + 16 < t.rows ? t.row0 + 16 : t.rows;
  seen(a, t, (int)p.share.div((uint32_t)t.row0), any_lo, all_hi);
  seen(a, t, (int)p.share.div((uint32_t)(row1 - 1)), all_lo, any_hi);

  // the steps that any row of the tile sees, of those that are this workgroup's
  const int s0 = any_lo / TOK > g0 ? any_lo / TOK : g0;
  const int s1 = any_hi <= any_lo ? s0 : (any_hi + TOK - 1) / TOK < g1 ? (any_hi + TOK - 1) / TOK : g1;
  const int stride = p.team ? kWaves : 1, step0 = p.team ? s0 + wave : s0, step1 = s1;

  char *rows = lds + wave * Shape::WAVE_BYTES;
  // A step's loads follow from its page numbers, so these are requested two steps
  // ahead, in front of the step's before: waiting for them then waits for no more
  // than what is used next.  All loads are unconditional, so that their number is
  // known; behind the part's end they repeat its last token.
  const int last_tok = (TOK * step1 < any_hi ? TOK * step1 : any_hi) - 1;
  auto token = [&](int step) {
    const int tok = TOK * step + (lane & (TOK - 1));
    return tok < last_tok ? tok : last_tok;
  };
  // Pages of whole steps: a step lies in one page, its rows are at fixed offsets from
  // one address; steps behind the part's end repeat its last.  (Together with the raw
  // registers' refill as they are used: 64 sequences 72 -> 62 us.)
  const bool whole = p.page.d % TOK == 0;
  // (without a table any word will do; the sequence's number stands for it)
  const int32_t *table = a.table ? a.table + (int64_t)t.b * a.table_pages : a.lengths + t.b;
  const uint32_t mask = a.table ? ~0u : 0u;
  auto entry = [&](int step) {
    const int tok = whole ? TOK * (step < step1 ? step : step1 - 1) : token(step);
    return table[p.page.div((uint32_t)tok) & mask];
  };
  const int64_t pages = a.cache.pages, heads = a.cache.heads;
  const uint32_t k_at = col * (HD / 2) + 4 * kg * W, ks_at = col * NB + kg * W / 4;
  auto load_k = [](const uint8_t *src, uint32_t (&k)[W]) {
    if constexpr (W == 4) {
      const u32x4 c = *(const u32x4 *)src;
#pragma unroll
      for (int e = 0; e < 4; e++) k[e] = c[e];
    } else if constexpr (W == 2) {
      const u32x2 c = *(const u32x2 *)src;
      k[0] = c[0], k[1] = c[1];
    } else {
      k[0] = *(const uint32_t *)src;
    }
  };
  auto load = [&](int step, int page, Raw<NB> &raw) {
    uint32_t pg, off;
    if (whole) {
      p.page.split((uint32_t)(TOK * (step < step1 ? step : step1 - 1)), pg, off);
      page = a.table ? uniform(page) : t.b;
      const bool there = (uint32_t)page < (uint64_t)pages;
      raw.missing = there ? 0 : ~0ull;
      const int64_t row = ((there ? page : 0) * heads + kh) * (int64_t)p.page.d + off;
      const uint8_t *kc = a.cache.k_codes + row * (HD / 2), *ks = a.cache.k_scales + row * NB;
      const uint8_t *vc = a.cache.v_codes + row * (HD / 2), *vs = a.cache.v_scales + row * NB;
#pragma unroll
      for (int i = 0; i < 2 * TS; i++)
#pragma unroll
        for (int j = 0; j < NL; j++) {
          // the lane's keys: elements 8 ((4 load + kg) W + dword) and the seven behind
          load_k(kc + (k_at + (16 * i * (HD / 2) + 16 * j * W)), raw.k[i][j]);
          raw.ks[i][j] = ks[ks_at + (16 * i * NB + j * W)];
        }
#pragma unroll
      for (int i = 0; i < NV; i++) {
        const uint32_t x = lane + 64 * i < TOK * NB ? lane + 64 * i : TOK * NB - 1;
        raw.v[i] = *(const u32x4 *)(vc + 16 * x);
        raw.vs[i] = vs[x];
      }
    } else {
      p.page.split((uint32_t)token(step), pg, off);
      page = a.table ? page : t.b;
      const bool there = (uint32_t)page < (uint64_t)pages;
      raw.missing = __ballot(!there);
      const int64_t row = ((there ? page : 0) * heads + kh) * (int64_t)p.page.d + off;
      const int rl = (int)row, rh = (int)(row >> 32);
      auto from = [&](int src) { return (int64_t)__shfl(rh, src) << 32 | (uint32_t)__shfl(rl, src); };
#pragma unroll
      for (int i = 0; i < 2 * TS; i++) {
        const int64_t at = from(16 * i + col);
#pragma unroll
        for (int j = 0; j < NL; j++) {
          load_k(a.cache.k_codes + at * (HD / 2) + 4 * (4 * j + kg) * W, raw.k[i][j]);
          raw.ks[i][j] = a.cache.k_scales[at * NB + (4 * j + kg) * W / 4];
        }
      }
#pragma unroll
      for (int i = 0; i < NV; i++) {
        const int x = lane + 64 * i, tok = x / NB < TOK ? x / NB : TOK - 1, blk = x % NB;
        const int64_t at = from(tok);
        raw.v[i] = *(const u32x4 *)(a.cache.v_codes + at * (HD / 2) + 16 * blk);
        raw.vs[i] = a.cache.v_scales[at * NB + blk];
      }
    }
  };

  Raw<NB> raw;
  int page = 0;
  if (step0 < step1) {
    const int now = entry(step0);
    page = entry(step0 + stride);
    load(step0, now, raw);
  }

  // the row of this lane's column, its tokens and operands; columns behind the last
  // row repeat it and see nothing
  int lo, hi;
  bf16x8 qf[NL * W][NQ];
  {
    const int r = t.row0 + col;
    uint32_t i, h;
    p.share.split((uint32_t)(r < t.rows ? r : t.rows - 1), i, h);
    seen(a, t, (int)i, lo, hi);
    if (r >= t.rows) lo = hi = 0;
    const T *q = (const T *)a.q + (t.start + (int64_t)i) * a.q_token + ((int64_t)kh * p.share.d + h) * a.q_head;
    float v[NL * W][8];
#pragma unroll
    for (int s = 0; s < NL * W; s++)  // step s = (load, dword): as the keys
      load8(q + 8 * ((4 * (s / W) + kg) * W + s % W), v[s]);
#pragma unroll
    for (int s = 0; s < NL * W; s++) {
      if (a.scale < 0.f)
#pragma unroll
        for (int k = 0; k < 8; k++) v[s][k] = -v[s][k];
      split8<NQ>(v[s], qf[s]);
    }
  }
  f32x4 o[2 * NB];
  float m = -kInf, l = 0.f;
#pragma unroll
  for (int d = 0; d < 2 * NB; d++) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto consume = [&](int step, Raw<NB> &cur) {
    // what is rare, out of the way: scales of NaN, pages that are not there, tokens
    // outside of what the tile sees.  Values that no row may meet become zeros (of
    // blocks of NaN below, what they make of the rows that see them).
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < NV; i++) odd = odd > cur.vs[i] ? odd : cur.vs[i];
#pragma unroll
    for (int i = 0; i < 2 * TS; i++)
#pragma unroll
      for (int j = 0; j < NL; j++) odd = odd > cur.ks[i][j] ? odd : cur.ks[i][j];
    uint64_t nan[NV] = {};
    uint64_t any_nan = 0;
    if (__any(kv_nan(odd)) || cur.missing || TOK * step < any_lo || TOK * step + TOK > any_hi) {
#pragma unroll
      for (int i = 0; i < NV; i++) {
        const int x = lane + 64 * i, tok = x / NB, at = TOK * step + tok;
        const bool in = tok < TOK && at >= any_lo && at < any_hi && !(cur.missing >> (tok & 63) & 1);
        nan[i] = __ballot(in && kv_nan(cur.vs[i]));
        any_nan |= nan[i];
        if (!in || kv_nan(cur.vs[i])) cur.v[i] = u32x4{0, 0, 0, 0}, cur.vs[i] = 127;
      }
#pragma unroll
      for (int i = 0; i < 2 * TS; i++)
#pragma unroll
        for (int j = 0; j < NL; j++)
          if (kv_nan(cur.ks[i][j]) || (cur.missing >> (16 * i + col) & 1)) cur.ks[i][j] = 255;
    }
    // values into the wave's LDS rows: behind the reads of the step before, as these are
    // of other lanes' writes (the hardware keeps a wave's LDS operations in their order,
    // the fences keep the compiler to it)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int x = lane + 64 * i, tok = x / NB, blk = x % NB;
      if (TOK * NB % 64 == 0 || tok < TOK)
#pragma unroll
        for (int c = 0; c < 4; c++)
          *(bf16x8 *)(rows + tok * ROWB + 64 * blk + 16 * (c ^ (tok & 3))) = fp4x8(cur.v[i][c], kv_scale(cur.vs[i]));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();

    f32x4 s[2 * TS];
#pragma unroll
    for (int i = 0; i < 2 * TS; i++) {
      s[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NL; j++) {
        const float sc = kv_scale(cur.ks[i][j]);
#pragma unroll
        for (int w = 0; w < W; w++) {
          const bf16x8 k = fp4x8(cur.k[i][j][w], sc);
#pragma unroll
          for (int n = NQ - 1; n >= 0; n--)  // small parts first
            s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, qf[j * W + w][n], s[i], 0, 0, 0);
        }
      }
    }
    // the step is in LDS and in the scores: its registers take the next loads
    __builtin_amdgcn_sched_barrier(0);
    const int now = page;
    page = entry(step + 2 * stride);
    load(step + stride, now, cur);
    __builtin_amdgcn_sched_barrier(0);
    // transposed reads: lanes 4j .. 4j+3 of 16 name token j's 16 elements
    const int j = col >> 2, c = col & 3;
    const char *vb = rows + (4 * kg + j) * ROWB + 8 * (c & 1);
    auto read = [&](int d, bf16x8 (&v)[TS]) {
#pragma unroll
      for (int h = 0; h < TS; h++) {
        const char *at = vb + 32 * h * ROWB + 64 * (d >> 1) + 16 * ((2 * (d & 1) + (c >> 1)) ^ j);
        const i16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)at);
        const i16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(at + 16 * ROWB));
        v[h] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    };
    // reads run two elements' blocks ahead of their products
    constexpr int AHEAD = 2;
    bf16x8 vt[AHEAD][TS];
#pragma unroll
    for (int d = 0; d < AHEAD; d++) read(d, vt[d]);

    float v[8 * TS];
#pragma unroll
    for (int e = 0; e < 8 * TS; e++) v[e] = s[e >> 2][e & 3];
    // tokens that not every row sees: rare, and a loop, which stays a branch
    int edges = uniform(TOK * step < all_lo || TOK * step + TOK > all_hi);
    asm volatile("" : "+s"(edges));
    for (; edges; edges = 0) {
      const int first = TOK * step + 4 * kg, a0 = lo - first, a1 = hi - first;
#pragma unroll
      for (int e = 0; e < 8 * TS; e++) {
        const int tok = 16 * (e >> 2) + (e & 3);
        if (tok < a0 || tok >= a1) v[e] = -kInf;
      }
    }
    float top = v[0];
#pragma unroll
    for (int e = 1; e < 8 * TS; e++) top = fmaxf(top, v[e]);
    top = fmaxf(m, max_over_16s(top) * p.log2_scale);
    // a row that sees nothing yet keeps -infinity; 0 stands for it here
    const float base = top == -kInf ? 0.f : top;
    if (__any(top > m)) {
      const float old = __builtin_amdgcn_exp2f(m - base);
      l *= old;
#pragma unroll
      for (int d = 0; d < 2 * NB; d++) o[d] *= old;
      m = top;
    }
#pragma unroll
    for (int e = 0; e < 8 * TS; e++) {
      v[e] = __builtin_amdgcn_exp2f(fmaf(v[e], p.log2_scale, -base));
      l += v[e];
    }
    // bf16 queries: weights rounded to bf16 (by 2^-8 of each at most), one product instead
    // of three; their sum l is of the fp32 ones
    bf16x8 pf[TS][NQ];
#pragma unroll
    for (int h = 0; h < TS; h++) split8<NQ>(v + 8 * h, pf[h]);
#pragma unroll
    for (int d = 0; d < 2 * NB; d++) {
#pragma unroll
      for (int h = 0; h < TS; h++)
#pragma unroll
        for (int n = NQ - 1; n >= 0; n--)
          o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt[d % AHEAD][h], pf[h][n], o[d], 0, 0, 0);
      if (d + AHEAD < 2 * NB) read(d + AHEAD, vt[d % AHEAD]);
    }
    if (any_nan) {
      // blocks of NaN among the values: NaN for the rows that see their tokens
#pragma unroll
      for (int i = 0; i < NV; i++) {
        for (uint64_t left = nan[i]; left; left &= left - 1) {
          const int x = __builtin_ctzll(left) + 64 * i, tok = TOK * step + x / NB, blk = x % NB;
#pragma unroll
          for (int d = 0; d < 2 * NB; d++)
            if (d >> 1 == blk && tok >= lo && tok < hi) o[d] += __builtin_nanf("");
        }
      }
    }
  };

  for (int step = step0; step < step1; step += stride) consume(step, raw);

  // elements d .. d + 3 of row r, finished or as a part
  auto emit = [&](int r, int d, f32x4 v, float top, float sum) {
    if (slot < 0) {
      uint32_t i, h;
      p.share.split((uint32_t)r, i, h);
      const int64_t tok = t.start + (int64_t)i, head = (int64_t)kh * p.share.d + h;
      if (sum == 0.f) v = f32x4{0.f, 0.f, 0.f, 0.f};
      else v *= 1.f / sum;
      store4((T *)a.out + tok * a.out_token + head * a.out_head + d, v);
      if (a.lse && d == 0) a.lse[tok * a.q_heads + head] = lse_of(top, sum);
    } else {
      const int64_t at = (int64_t)slot * p.rows + (r - t.row0);
      if (d == 0) p.part_ml[at] = f32x2{top, sum};
      if (sum != 0.f) *(f32x4 *)(p.part + at * HD + d) = v;
    }
  };
  l = sum_over_16s(l);
  if (!p.team) {
    const int r = t.row0 + col;
    if (r < t.rows)
#pragma unroll
      for (int d = 0; d < 2 * NB; d++) emit(r, 16 * d + 4 * kg, o[d], m, l);
    continue;
  }
  // the team's sums, in the order of its waves, through their LDS
  auto ml = [&](int w, int c) -> f32x2 & {
    return *(f32x2 *)(lds + w * Shape::WAVE_BYTES + 16 * Shape::OSTRIDE * 4 + 8 * c);
  };
#pragma unroll
  for (int d = 0; d < 2 * NB; d++) *(f32x4 *)((float *)rows + col * Shape::OSTRIDE + 16 * d + 4 * kg) = o[d];
  if (kg == 0) ml(wave, col) = f32x2{m, l};
  __syncthreads();
  for (int e = tid; e < 16 * (HD / 4); e += 64 * kWaves) {
    const int c = e / (HD / 4), d = 4 * (e % (HD / 4)), r = t.row0 + c;
    if (r >= t.rows) break;
    float top = ml(0, c)[0], sum = 0.f;
#pragma unroll
    for (int w = 1; w < kWaves; w++) top = fmaxf(top, ml(w, c)[0]);
    const float base = top == -kInf ? 0.f : top;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
      const float f = __builtin_amdgcn_exp2f(ml(w, c)[0] - base);
      sum += ml(w, c)[1] * f;
      v += *(const f32x4 *)(lds + w * Shape::WAVE_BYTES + (c * Shape::OSTRIDE + d) * 4) * f;
    }
    emit(r, d, v, top, sum);
  }
  __syncthreads();  // the LDS is free again
  }
}

template <int NB>
void launch(const KvLaunch &p, dim3 grid) {
  if (p.a.dtype == 0) hipLaunchKernelGGL((kv_rows_kernel<NB, true>), grid, dim3(256), 0, p.a.stream, p);
  else hipLaunchKernelGGL((kv_rows_kernel<NB, false>), grid, dim3(256), 0, p.a.stream, p);
}

}  // namespace

hipError_t launch_kv_rows(const KvLaunch &p) {
  const dim3 grid(p.team ? (unsigned)p.workers : (unsigned)((p.workers ? p.workers : p.count) + kWaves - 1) / kWaves,
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
