// kv_attention_tiles.hip -- attention of many rows (chunks, prompts) over the
// 4-bit cache.
//
// A workgroup takes a tile of rows, 32 for each of its waves, and walks over the
// tokens 64 a step.  The step's keys and values are converted once for all waves, into
// LDS as bf16 (two buffers: the next step's are written while this one's are read).  A wave computes
//   S^T = K Q^T   and   O^T = V^T P^T
// with 32x32x16 matrix instructions; the first leaves each lane eight tokens of its
// row a time, in an order that the second takes as its operand, so the weights
// never leave their lane.  V^T comes from LDS by transposed reads.  16-byte pieces
// of a row are swizzled by the token, so that neither the operands' reads nor the
// conversion's writes conflict.
//
// Bound by the matrix unit and the instructions beside it: 1560 queries over 32760
// tokens, 40 heads of 128, bf16, 1.05 TFLOP, 1.15 to 1.16 ms with the join (0.91 PFLOP/s; a
// large product of the library reaches 1.3 to 1.6).  That is 6 tiles of 256 rows and one
// of 24, whose waves without rows work as the others do: 13% of the products.
// Four waves of twice 32 rows 1.87 ms; operands read as the compiler orders them 1.21 ms;
// two groups of waves half a step apart, or the scores of the next step computed beside
// this one's weights within a wave, no faster (1.23).
// Causal prompts of 4096 and 8192 tokens, 32 query and 8 key heads: 255 and 730 us.
// fp32 heads of 192 / 224 / 256 (71 / 263 / 383 registers) and bf16 heads of 256 (41)
// spill: a prompt of 2048 tokens, heads of 128, 192, 256, takes 80, 176, 253 us in bf16 and
// 213, 381, 1175 us in fp32.
#include <hip/hip_runtime.h>

#include "kv_attention.h"

namespace oq {
namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
typedef __attribute__((address_space(3))) const bf16x8 lds_bf16x8;
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kTok = kKvTilesStep;

// A token's row in LDS: 4 NB pieces of 16 bytes.  Rows repeat their banks every
// 256 bytes, that is every 1, 2 or 4 tokens by NB modulo 4; the piece's number is
// changed by the bits of the token that the row's place does not use, so that any
// 16 tokens in line (16-byte reads of one piece) and any four (8-byte reads of four
// pieces) meet all banks alike.
template <int NB>
__device__ __forceinline__ int swizzle(int tok) {
  constexpr int HIGH = NB % 4 == 0 ? 2 : NB % 2 == 0 ? 1 : 0;
  return ((tok & 3) >> (2 - HIGH) << 2) | (tok >> 2 & 3);
}

// Scores of tokens outside [a0, a1) (counted from the lane's first) to -infinity.
// Rare: the empty asm keeps the compiler from doing it every time.
__device__ __forceinline__ void hide(f32x16 &s, int a0, int a1) {
#pragma unroll
  for (int e = 0; e < 16; e++) {
    const int tok = (e & 3) + 8 * (e >> 2);
    float v = tok < a0 || tok >= a1 ? -kInf : s[e];
    asm volatile("" : "+v"(v));
    s[e] = v;
  }
}

template <int NB, int WAVES, bool F32>
__global__ __launch_bounds__(64 * WAVES, WAVES / 4) void kv_tiles_kernel(KvLaunch p) {
  using T = typename std::conditional<F32, float, uint16_t>::type;
  constexpr int HD = 32 * NB, ROWB = 2 * HD, NQ = F32 ? 3 : 1, TASKS = (2 * NB + WAVES - 1) / WAVES;
  __shared__ __attribute__((aligned(16))) char lds[2][2][kTok * ROWB];  // [buffer][keys, values]
  __shared__ int nans[4];  // by step modulo 4: blocks of NaN among the values
  constexpr int AHEAD = 4;
  const KvAttentionArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, half = lane >> 5;
  const int wave = uniform(tid >> 6);
  int share = 0, pos = 0, end = 1;
  KvUnits u;
  if (p.workers) u = first_units(p, blockIdx.x, share, pos, end);
  for (bool again = false; pos < end; again = true) {
    // the group, and this workgroup's steps of it
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
      if (len < u.units) slot = 2 * (int)blockIdx.x + (skip == 0);
      if (skip == 0 && tid == 0)
        p.parts[(int64_t)(u.tiles_before + tile) * a.cache.heads + kh] =
            int2{slot, (pos + u.units - 1) / share - (int)blockIdx.x + 1};
      pos += len;
    } else {
      t = find_tile(p, blockIdx.x);
      kh = blockIdx.y;
      pos = end;
      if (t.b < 0) return;
    }
    t = uniform(t), kh = uniform(kh), g0 = uniform(g0), g1 = uniform(g1), slot = uniform(slot), pos = uniform(pos);
    // what the tile as a whole sees, and what every row of it sees
    int any_lo, any_hi, all_lo, all_hi;
    const int row1 = t.row0 + p.rows < t.rows ? t.row0 + p.rows : t.rows;
    seen(a, t, (int)p.share.div((uint32_t)t.row0), any_lo, all_hi);
    seen(a, t, (int)p.share.div((uint32_t)(row1 - 1)), all_lo, any_hi);
    const int step0 = any_lo / kTok > g0 ? any_lo / kTok : g0;
    const int step1 = any_hi <= any_lo ? step0 : (any_hi + kTok - 1) / kTok < g1 ? (any_hi + kTok - 1) / kTok : g1;

    // Conversion: task x of a step is block x % NB of token x / NB, first of the keys,
    // then of the values; a thread has TASKS of them, a wave's all of one kind.
    const int last_tok = (kTok * step1 < any_hi ? kTok * step1 : any_hi) - 1;
    const int32_t *table = a.table ? a.table + (int64_t)t.b * a.table_pages : a.lengths + t.b;
    const uint32_t mask = a.table ? ~0u : 0u;
    auto values = [&](int i) { return wave + WAVES * i >= NB; };
    auto task = [&](int i) {
      const int x = tid + 64 * WAVES * i;
      return x < kTok * NB ? x : x < 2 * kTok * NB ? x - kTok * NB : kTok * NB - 1;
    };
    auto token = [&](int step, int i) {
      const int tok = kTok * step + task(i) / NB;
      return tok < last_tok ? tok : last_tok;
    };
    auto entry = [&](int step, int (&page)[TASKS]) {
#pragma unroll
      for (int i = 0; i < TASKS; i++) page[i] = table[p.page.div((uint32_t)token(step, i)) & mask];
    };
    struct Raw {
      u32x4 c[TASKS];
      uint32_t s[TASKS];
      bool missing[TASKS];
    };
    const int64_t pages = a.cache.pages, heads = a.cache.heads;
    auto load = [&](int step, const int (&page)[TASKS], Raw &raw) {
#pragma unroll
      for (int i = 0; i < TASKS; i++) {
        uint32_t pg, off;
        p.page.split((uint32_t)token(step, i), pg, off);
        const int n = a.table ? page[i] : t.b;
        raw.missing[i] = (uint32_t)n >= (uint64_t)pages;
        const int64_t row = ((raw.missing[i] ? 0 : n) * heads + kh) * (int64_t)p.page.d + off;
        const int64_t at = row * NB + task(i) % NB;
        raw.c[i] = *(const u32x4 *)((values(i) ? a.cache.v_codes : a.cache.k_codes) + 16 * at);
        raw.s[i] = (values(i) ? a.cache.v_scales : a.cache.k_scales)[at];
      }
    };
    // A step's keys and values into a buffer.  A thread's four pieces go out in an
    // order of its own (its dwords are exchanged by two bits of the token), so that
    // neighbours write to different banks.
    auto convert = [&](int step, Raw &raw, int buffer) {
#pragma unroll
      for (int i = 0; i < TASKS; i++) {
        if (wave + WAVES * i >= 2 * NB) break;
        const int x = task(i), tok = x / NB, blk = x % NB, at = kTok * step + tok;
        const bool nan = kv_nan(raw.s[i]);
        if (values(i)) {
          if (at < any_lo || at >= any_hi || raw.missing[i]) raw.c[i] = u32x4{0, 0, 0, 0}, raw.s[i] = 127;
          else if (nan) raw.c[i] = u32x4{0, 0, 0, 0}, raw.s[i] = 127, nans[step & 3] = 1;  // put right behind the products
        } else if (nan || raw.missing[i]) {
          raw.s[i] = 255;
        }
        const float scale = kv_scale(raw.s[i]);
        const bool b0 = tok & 1, b1 = tok & 2;
        u32x4 w = raw.c[i];
        w = u32x4{b0 ? w[1] : w[0], b0 ? w[0] : w[1], b0 ? w[3] : w[2], b0 ? w[2] : w[3]};
        w = u32x4{b1 ? w[2] : w[0], b1 ? w[3] : w[1], b1 ? w[0] : w[2], b1 ? w[1] : w[3]};
        char *row = &lds[buffer][values(i)][tok * ROWB];
        const int sw = swizzle<NB>(tok);
#pragma unroll
        for (int c = 0; c < 4; c++)
          *(bf16x8 *)(row + 16 * ((4 * blk + (c ^ (tok & 3))) ^ sw)) = fp4x8(w[c], scale);
      }
    };

    Raw raw;
    int page[TASKS];
    __syncthreads();  // the buffers and flags of the group before are read
    if (tid < 4) nans[tid] = 0;
    if (step0 < step1) {
      int first[TASKS];
      entry(step0, first);
      entry(step0 + 1, page);
      load(step0, first, raw);
    }

    // the row of this lane's column, its tokens and operands; columns behind the last
    // row repeat it and see nothing
    int lo, hi;
    bf16x8 qf[HD / 16][NQ];
    {
      const int r = t.row0 + 32 * wave + col;
      uint32_t i, h;
      p.share.split((uint32_t)(r < t.rows ? r : t.rows - 1), i, h);
      seen(a, t, (int)i, lo, hi);
      if (r >= t.rows) lo = hi = 0;
      const T *q = (const T *)a.q + (t.start + (int64_t)i) * a.q_token + ((int64_t)kh * p.share.d + h) * a.q_head;
#pragma unroll
      for (int s = 0; s < HD / 16; s++) {
        float v[8];
        load8(q + 16 * s + 8 * half, v);
        if (a.scale < 0.f)
#pragma unroll
          for (int k = 0; k < 8; k++) v[k] = -v[k];
        split8<NQ>(v, qf[s]);
      }
    }
    f32x16 o[NB];
    float m = -kInf, l = 0.f;
#pragma unroll
    for (int d = 0; d < NB; d++)
#pragma unroll
      for (int e = 0; e < 16; e++) o[d][e] = 0.f;
    // LDS addresses of the operands' reads: of keys a row a lane, of values (transposed:
    // lanes 4j .. 4j+3 of 16 name token j's 16 elements) rows j and j + 8 of 16.  They
    // change from buffer to buffer with the step; 16 and 32 tokens on is an offset, as
    // the swizzle is the same there.
    constexpr uint32_t BUFFER = 2 * kTok * ROWB;
    uint32_t k_at[HD / 16], v_at[NB][2];
    {
      const uint32_t base = (uint32_t)(uintptr_t)(lds_char *)&lds[0][0][0] + (step0 & 1) * BUFFER;
#pragma unroll
      for (int c = 0; c < HD / 16; c++) k_at[c] = base + col * ROWB + 16 * ((2 * c + half) ^ swizzle<NB>(col));
      const int c = lane & 3, which = lane >> 4 & 1;
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const int tok = 4 * half + ((lane & 15) >> 2) + 8 * k;
#pragma unroll
        for (int d = 0; d < NB; d++)
          v_at[d][k] = base + kTok * ROWB + tok * ROWB + 16 * ((4 * d + 2 * which + (c >> 1)) ^ swizzle<NB>(tok)) + 8 * (c & 1);
      }
    }
    __syncthreads();  // the flags are clear
    if (step0 < step1) {
      convert(step0, raw, step0 & 1);
      load(step0 + 1, page, raw);
      entry(step0 + 2, page);
    }

    for (int step = step0; step < step1; step++) {
      __syncthreads();  // this step's buffer is written, the other one read
      const int buffer = step & 1;
      if (step + 1 < step1) {
        convert(step + 1, raw, buffer ^ 1);
        load(step + 2, page, raw);
        entry(step + 3, page);
      }
      if (tid == 0) nans[(step + 3) & 3] = 0;
      // Reads run AHEAD products ahead, in this order: left to itself the compiler waits
      // for each.
      f32x16 s[2];
#pragma unroll
      for (int i = 0; i < 2; i++)
#pragma unroll
        for (int e = 0; e < 16; e++) s[i][e] = 0.f;
      auto key = [&](int c) { return *(lds_bf16x8 *)(uintptr_t)(k_at[c % (HD / 16)] + c / (HD / 16) * 32 * ROWB); };
      bf16x8 kf[AHEAD];
#pragma unroll
      for (int c = 0; c < AHEAD; c++) kf[c] = key(c);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = 0; c < HD / 8; c++) {
        f32x16 &to = s[c / (HD / 16)];
#pragma unroll
        for (int n = NQ - 1; n >= 0; n--)  // small parts first
          to = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[c % AHEAD], qf[c % (HD / 16)][n], to, 0, 0, 0);
        if (c + AHEAD < HD / 8) kf[c % AHEAD] = key(c + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
      }
      // product x of the second: token 16 (x / NB), elements 32 (x % NB)
      auto value = [&](int x) {
        const uint32_t on = x / NB * 16 * ROWB;
        const i16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(uintptr_t)(v_at[x % NB][0] + on));
        const i16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(uintptr_t)(v_at[x % NB][1] + on));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
      };
      bf16x8 vf[AHEAD];
#pragma unroll
      for (int c = 0; c < AHEAD; c++) vf[c] = value(c);
      __builtin_amdgcn_sched_barrier(0);
      if (kTok * step < all_lo || kTok * step + kTok > all_hi) {
        const int first = kTok * step + 4 * half;
        hide(s[0], lo - first, hi - first);
        hide(s[1], lo - first - 32, hi - first - 32);
      }
      // (the instruction that keeps a NaN: a row with one is NaN, and it takes three)
      float top = __builtin_elementwise_maximum(s[0][0], s[1][0]);
#pragma unroll
      for (int e = 1; e < 16; e++)
        top = __builtin_elementwise_maximum(__builtin_elementwise_maximum(top, s[0][e]), s[1][e]);
      const uint32_t tb = __float_as_uint(top);
      const auto other = __builtin_amdgcn_permlane32_swap(tb, tb, false, false);
      top = fmaxf(__uint_as_float(other[0]), __uint_as_float(other[1])) * p.log2_scale;
      // the maximum follows only where weights could pass 2^8: they keep their relative
      // accuracy up to there
      if (__any(top > m + 8.f)) {
        top = fmaxf(m, top);
        const float old = __builtin_amdgcn_exp2f(m - (top == -kInf ? 0.f : top));
        l *= old;
#pragma unroll
        for (int d = 0; d < NB; d++) o[d] *= old;
        m = top;
      }
      // a row that sees nothing yet keeps -infinity; 0 stands for it here
      const float base = m == -kInf ? 0.f : m;
      // the second 32 tokens' weights between the first's products
      float v[2][16];
      // (bf16 queries: weights rounded to bf16, by 2^-8 of each at most, one product instead
      // of three; their sum l is of the fp32 ones.  Error of this frame's outputs against 64
      // bits 0.0019, with fp32 weights 0.0016, which is the outputs' own rounding.)
      bf16x8 pf[4][NQ];
      auto weigh = [&](int i, int e) {
        v[i][e] = __builtin_amdgcn_exp2f(fmaf(s[i][e], p.log2_scale, -base));
        l += v[i][e];
      };
#pragma unroll
      for (int e = 0; e < 16; e++) weigh(0, e);
      split8<NQ>(v[0], pf[0]);
      split8<NQ>(v[0] + 8, pf[1]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int x = 0; x < 4 * NB; x++) {
#pragma unroll
        for (int n = NQ - 1; n >= 0; n--)
          o[x % NB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[x % AHEAD], pf[x / NB][n], o[x % NB], 0, 0, 0);
        if (x + AHEAD < 4 * NB) vf[x % AHEAD] = value(x + AHEAD);
        if (x < 2 * NB) {
          constexpr int EACH = (16 + 2 * NB - 1) / (2 * NB);
#pragma unroll
          for (int e = EACH * x; e < EACH * (x + 1) && e < 16; e++) weigh(1, e);
          if (x == 2 * NB - 1) {
            split8<NQ>(v[1], pf[2]);
            split8<NQ>(v[1] + 8, pf[3]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int c = 0; c < HD / 16; c++) k_at[c] += buffer ? -BUFFER : BUFFER;
#pragma unroll
      for (int d = 0; d < NB; d++) v_at[d][0] += buffer ? -BUFFER : BUFFER, v_at[d][1] += buffer ? -BUFFER : BUFFER;
      if (uniform(nans[step & 3])) {
        // blocks of NaN among the values: NaN for the rows that see their tokens
        for (int tok = kTok * step; tok < kTok * step + kTok; tok++) {
          if (tok < any_lo || tok >= any_hi) continue;
          uint32_t pg, off;
          p.page.split((uint32_t)tok, pg, off);
          const int n = a.table ? table[pg] : t.b;
          if ((uint32_t)n >= (uint64_t)pages) continue;
          const int64_t row = (n * heads + kh) * (int64_t)p.page.d + off;
#pragma unroll
          for (int d = 0; d < NB; d++)
            if (kv_nan(a.cache.v_scales[row * NB + d]) && tok >= lo && tok < hi)
              o[d] += __builtin_nanf("");
        }
      }
    }

    const int r = t.row0 + 32 * wave + col;
    const uint32_t lb = __float_as_uint(l);
    const auto other = __builtin_amdgcn_permlane32_swap(lb, lb, false, false);
    const float sum = __uint_as_float(other[0]) + __uint_as_float(other[1]);
    if (r < t.rows) {
      uint32_t i, h;
      p.share.split((uint32_t)r, i, h);
      const int64_t tok = t.start + (int64_t)i, head = (int64_t)kh * p.share.d + h;
      const int64_t at = (int64_t)slot * p.rows + (r - t.row0);
      const float inv = 1.f / sum;
#pragma unroll
      for (int d = 0; d < NB; d++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          f32x4 v = {o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
          const int el = 32 * d + 8 * e + 4 * half;
          if (slot < 0)
            store4((T *)a.out + tok * a.out_token + head * a.out_head + el,
                   sum == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : v * inv);
          else if (sum != 0.f)
            *(f32x4 *)(p.part + at * HD + el) = v;
        }
      if (half == 0) {
        if (slot >= 0) p.part_ml[at] = f32x2{m, sum};
        else if (a.lse) a.lse[tok * a.q_heads + head] = lse_of(m, sum);
      }
    }
  }
}

template <int NB>
void launch(const KvLaunch &p, dim3 grid) {
  constexpr int W16 = kv_tiles_rows(1, 32 * NB) / 32, W32 = kv_tiles_rows(0, 32 * NB) / 32;
  if (p.a.dtype == 1) hipLaunchKernelGGL((kv_tiles_kernel<NB, W16, false>), grid, dim3(64 * W16), 0, p.a.stream, p);
  else hipLaunchKernelGGL((kv_tiles_kernel<NB, W32, true>), grid, dim3(64 * W32), 0, p.a.stream, p);
}

}  // namespace

hipError_t launch_kv_tiles(const KvLaunch &p) {
  const dim3 grid(p.workers ? (unsigned)p.workers : (unsigned)p.count, p.workers ? 1u : (unsigned)p.a.cache.heads);
  switch (p.a.cache.head_dim / 32) {
#define OQ_CASE(NB) \
  case NB: launch<NB>(p, grid); break;
    OQ_CASE(1) OQ_CASE(2) OQ_CASE(3) OQ_CASE(4) OQ_CASE(5) OQ_CASE(6) OQ_CASE(7) OQ_CASE(8)
#undef OQ_CASE
  }
  return hipGetLastError();
}

}  // namespace oq
