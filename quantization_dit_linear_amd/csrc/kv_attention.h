// kv_attention.h -- what the kernels of attention over the 4-bit cache share.
#pragma once
#include <hip/hip_runtime.h>

#include "kv_cache.h"
#include "mx_codec.h"
#include "oq_internal.h"

namespace oq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kInf = __builtin_huge_valf();
constexpr float kLn2 = 0.6931471805599453f;

// One launch.  A group is a tile of `rows` (query, head of the group) rows of a
// sequence with one key head; its units are steps of `step` tokens, and `extra` in
// front that stand for the time a group takes besides.
// workers = 0: a wave a group.  Otherwise `workers` waves (team: workgroups, whose
// waves take the steps by turns) share all units evenly: each takes the next of the
// order (sequence, key head, tile, step), and where that cuts a group, its parts go
// to the workspace, to be joined in their order.
struct KvLaunch {
  KvAttentionArgs a;
  FastDiv page, share, tiles;  // share: heads of a key head; tiles: of a sequence, where all have as many queries
  int rows, step, extra;
  int count, workers, least;  // count: tiles (at most); least: units of a worker
  int each;                   // queries of a sequence, where all have as many
  bool team;
  float log2_scale;           // |scale| log2 e; a negative scale turns the queries
  float *part;     // [2 workers][rows][head_dim]: a worker's first part, then its last
  f32x2 *part_ml;  // [2 workers][rows]: maximum (log2), sum of weights
  int2 *parts;     // [tiles][heads]: a group's first part, and their number
};

// The rows of one tile.
struct KvTile {
  int b;       // sequence, -1: none
  int row0;    // first row in the sequence
  int rows;    // rows of the sequence (queries times heads of the group)
  int start;   // the sequence's first token of q
  int n;       // queries
  int length;  // tokens in the cache
};

__device__ __forceinline__ int clamped(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// Sequence b's queries and length.
__device__ __forceinline__ KvTile sequence(const KvLaunch &p, int b) {
  const KvAttentionArgs &a = p.a;
  KvTile t;
  t.b = b, t.row0 = 0;
  if (a.q_starts) {
    const int most = (int)a.q_tokens;
    t.start = clamped(a.q_starts[b], 0, most);
    t.n = clamped(a.q_starts[b + 1], t.start, most) - t.start;
  } else {
    t.n = p.each;
    t.start = b * t.n;
  }
  t.rows = t.n * (int)p.share.d;
  t.length = clamped(a.lengths[b], 0, a.table_pages * a.cache.page);
  return t;
}

// The inclusive sum over the lanes up to this one: within rows of 16 lanes, then
// each row's last lane into the rows behind it.
__device__ __forceinline__ int prefix_sum(int v) {
#define OQ_STEP(CTRL, ROWS) v += __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false)
  OQ_STEP(0x111, 0xf);  // the lane before
  OQ_STEP(0x112, 0xf);
  OQ_STEP(0x114, 0xf);
  OQ_STEP(0x118, 0xf);
  OQ_STEP(0x142, 0xa);  // lane 15 of the row before, into rows 1 and 3
  OQ_STEP(0x143, 0xc);  // lane 31 into rows 2 and 3
#undef OQ_STEP
  return v;
}

// The same, known to be the same in all lanes.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ KvTile uniform(KvTile t) {
  return {uniform(t.b), uniform(t.row0), uniform(t.rows), uniform(t.start), uniform(t.n), uniform(t.length)};
}

__device__ __forceinline__ KvTile from_lane(KvTile t, int l) {
  return {__builtin_amdgcn_readlane(t.b, l), __builtin_amdgcn_readlane(t.row0, l), __builtin_amdgcn_readlane(t.rows, l),
          __builtin_amdgcn_readlane(t.start, l), __builtin_amdgcn_readlane(t.n, l), __builtin_amdgcn_readlane(t.length, l)};
}

// Tile x of the launch.  Sequences of their own lengths: 64 of them at a time, a
// prefix sum of their tiles over the wave's lanes (every wave for itself).
__device__ __forceinline__ KvTile find_tile(const KvLaunch &p, int x) {
  const int lane = threadIdx.x & 63;
  if (!p.a.q_starts) {
    uint32_t b, r;
    p.tiles.split((uint32_t)x, b, r);
    KvTile t = sequence(p, (int)b);
    t.row0 = (int)r * p.rows;
    return t;
  }
  for (int b0 = 0, before = 0; b0 < p.a.batch; b0 += 64) {
    KvTile t{-1, 0, 0, 0, 0, 0};
    if (b0 + lane < p.a.batch) t = sequence(p, b0 + lane);
    const int tiles = (t.rows + p.rows - 1) / p.rows, sum = before + prefix_sum(tiles);
    const uint64_t past = __ballot(sum > x);
    if (past) {
      const int l = __builtin_ctzll(past);
      t.row0 = (x - sum + tiles) * p.rows;
      return from_lane(t, l);
    }
    before = __builtin_amdgcn_readlane(sum, 63);
  }
  return {-1, 0, 0, 0, 0, 0};
}

// The tokens [lo, hi) that query i of a tile's sequence sees.
__device__ __forceinline__ void seen(const KvAttentionArgs &a, const KvTile &t, int i, int &lo, int &hi) {
  lo = 0, hi = t.length;
  if (a.causal) {
    const int at = t.length - t.n + i + 1;  // tokens up to the query's own
    hi = at < 0 ? 0 : at < hi ? at : hi;
    if (a.window && at > a.window) lo = at - a.window;
    if (lo > hi) lo = hi;
  }
}

// A sequence in the order of the units: every (key head, tile) of it has `units`,
// the last of them steps of the cache from step `first`.
struct KvUnits {
  KvTile t;
  int before, tiles_before;  // units and tiles of the sequences before
  int tiles, units, first;
  __device__ int all(int heads) const { return heads * tiles * units; }
};

__device__ __forceinline__ KvUnits units_of(const KvLaunch &p, int b) {
  KvUnits u{{-1, 0, 0, 0, 0, 0}, 0, 0, 0, 0, 0};
  if (b >= p.a.batch) return u;
  u.t = sequence(p, b);
  if (u.t.n == 0) return u;
  u.tiles = (u.t.rows + p.rows - 1) / p.rows;
  int lo, hi, unused;
  seen(p.a, u.t, 0, lo, unused);
  seen(p.a, u.t, u.t.n - 1, unused, hi);
  u.first = lo / p.step;
  u.units = (hi + p.step - 1) / p.step - u.first;
  u.units = p.extra + (u.units < 0 ? 0 : u.units);  // (rows that see nothing are written too)
  return u;
}

// The sequence that unit x belongs to (none past the last), among the 64 from b0 on
// of which the lanes hold one each, all its units and the prefix sums of these and of
// the tiles.
__device__ __forceinline__ KvUnits pick(const KvUnits &u, int all, int sum, int tsum, uint64_t past) {
  const int l = __builtin_ctzll(past);
  return {from_lane(u.t, l),
          __builtin_amdgcn_readlane(sum - all, l),
          __builtin_amdgcn_readlane(tsum - u.tiles, l),
          __builtin_amdgcn_readlane(u.tiles, l),
          __builtin_amdgcn_readlane(u.units, l),
          __builtin_amdgcn_readlane(u.first, l)};
}

// The sequence that unit x belongs to (x below the total).
__device__ __forceinline__ KvUnits find_units(const KvLaunch &p, int x) {
  const int lane = threadIdx.x & 63;
  for (int b0 = 0, before = 0, tiles = 0; b0 < p.a.batch; b0 += 64) {
    const KvUnits u = units_of(p, b0 + lane);
    const int all = u.all(p.a.cache.heads), sum = before + prefix_sum(all), tsum = tiles + prefix_sum(u.tiles);
    const uint64_t past = __ballot(sum > x);
    if (past) return pick(u, all, sum, tsum, past);
    before = __builtin_amdgcn_readlane(sum, 63);
    tiles = __builtin_amdgcn_readlane(tsum, 63);
  }
  return {{-1, 0, 0, 0, 0, 0}, 0, 0, 0, 0, 0};
}

// A worker's units [pos, end), `share` each, and the sequence of the first.
__device__ __forceinline__ KvUnits first_units(const KvLaunch &p, int worker, int &share, int &pos, int &end) {
  const int lane = threadIdx.x & 63;
  int total = 0, tiles = 0;
  KvUnits u;
  int all = 0, sum = 0, tsum = 0;
  for (int b0 = 0; b0 < p.a.batch; b0 += 64) {
    u = units_of(p, b0 + lane);
    all = u.all(p.a.cache.heads);
    sum = prefix_sum(all), tsum = prefix_sum(u.tiles);
    total += __builtin_amdgcn_readlane(sum, 63);
    tiles += __builtin_amdgcn_readlane(tsum, 63);
    // starts that descend name tokens twice and can make more tiles than the sizes
    // allow, which the workspace has no place for: then no worker does anything
    if (tiles > p.count) {
      total = 0;
      break;
    }
  }
  share = (total + p.workers - 1) / p.workers;
  if (share < p.least) share = p.least;
  pos = worker * share;
  end = pos + share < total ? pos + share : total;
  if (pos >= end) return u;
  if (p.a.batch > 64) return find_units(p, pos);
  return pick(u, all, sum, tsum, __ballot(sum > pos));
}

// Eight e2m1 codes of one block as bf16: exact at every scale.
__device__ __forceinline__ bf16x8 fp4x8(uint32_t w, float scale) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const b2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const b2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const b2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// Scale bytes that attention reads as NaN: the writer's 255, and those whose
// blocks could pass bf16's range.  255 as an exponent makes the conversion's
// results NaN; 0 its results subnormal or zero.
__device__ __forceinline__ bool kv_nan(uint32_t s) { return s >= 253; }
__device__ __forceinline__ float kv_scale(uint32_t s) { return __uint_as_float(s << 23); }

// Eight fp32 values as bf16 in NQ parts whose sum they are: one, rounded to
// nearest, or three, which hold all 24 bits.
template <int NQ>
__device__ __forceinline__ void split8(const float *v, bf16x8 *out) {
#pragma unroll
  for (int e = 0; e < 8; e++) {
    float x = v[e];
#pragma unroll
    for (int k = 0; k < NQ; k++) {
      out[k][e] = (__bf16)x;
      if (k + 1 < NQ) x -= (float)out[k][e];
    }
  }
}

// max and sum over the lanes that differ in bits 4 and 5
__device__ __forceinline__ float max_over_16s(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint32_t w = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_16s(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const uint32_t w = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Four consecutive elements of a finished row.
template <class T>
__device__ __forceinline__ void store4(T *p, f32x4 v) {
  if constexpr (sizeof(T) == 2) {
    const bf16x2 a = {(__bf16)v[0], (__bf16)v[1]}, b = {(__bf16)v[2], (__bf16)v[3]};
    *(u32x2 *)p = u32x2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
  } else {
    *(f32x4 *)p = v;
  }
}

__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -kInf : (m + log2f(l)) * kLn2; }

// tokens a step of the rows kernel
constexpr int kv_rows_step(int head_dim) { return head_dim <= 128 ? 64 : 32; }
hipError_t launch_kv_rows(const KvLaunch &p);
// rows of a workgroup's tile and tokens a step of the tiles kernel
constexpr int kv_tiles_rows(int dtype, int head_dim) { return head_dim > (dtype == 0 ? 64 : 128) ? 128 : 256; }
constexpr int kKvTilesStep = 64;
hipError_t launch_kv_tiles(const KvLaunch &p);

}  // namespace oq
