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

// One launch: tiles of `rows` (query, head of the group) rows of a sequence, in
// the order of the sequences, times the key heads, times `splits` parts of the
// tokens.  With more than one part every row leaves its sum, maximum and sum of
// weights in the workspace, and the join adds the parts up in their order.
struct KvLaunch {
  KvAttentionArgs a;
  FastDiv page, share, tiles;  // tiles: of a sequence, where all have as many queries
  int rows, splits;
  float log2_scale;            // |scale| log2 e; a negative scale turns the queries
  float *part;                 // [splits][q_tokens][q_heads][head_dim]
  f32x2 *part_ml;              // [splits][q_tokens][q_heads]: maximum (log2), sum
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

// Tile x of the launch.  Sequences of their own lengths: 64 of them at a time, a
// prefix sum of their tiles over the wave's lanes (every wave for itself).
__device__ __forceinline__ KvTile find_tile(const KvLaunch &p, int x) {
  const KvAttentionArgs &a = p.a;
  KvTile t{-1, 0, 0, 0, 0, 0};
  int tile = 0;
  if (!a.q_starts) {
    uint32_t b, r;
    p.tiles.split((uint32_t)x, b, r);
    t.b = (int)b, tile = (int)r;
    t.n = (int)(a.q_tokens / a.batch);
    t.start = t.b * t.n;
  } else {
    const int lane = threadIdx.x & 63, share = (int)p.share.d, most = (int)a.q_tokens;
    int before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
      const int b = b0 + lane;
      int s = 0, n = 0;
      if (b < a.batch) {
        s = clamped(a.q_starts[b], 0, most);
        n = clamped(a.q_starts[b + 1], s, most) - s;
      }
      const int tiles = (n * share + p.rows - 1) / p.rows;
      int sum = tiles;
#pragma unroll
      for (int off = 1; off < 64; off *= 2) {
        const int o = __shfl_up(sum, off);
        if (lane >= off) sum += o;
      }
      const uint64_t past = __ballot(before + sum > x);
      if (past) {
        const int l = __builtin_ctzll(past);
        t.b = b0 + l;
        t.start = __builtin_amdgcn_readlane(s, l);
        t.n = __builtin_amdgcn_readlane(n, l);
        tile = x - before - (__builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(tiles, l));
        break;
      }
      before += __builtin_amdgcn_readlane(sum, 63);
    }
    if (t.b < 0) return t;
  }
  t.row0 = tile * p.rows;
  t.rows = t.n * (int)p.share.d;
  t.length = clamped(a.lengths[t.b], 0, a.table_pages * a.cache.page);
  return t;
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

// The cache row of token t (of its key head) in sequence b; -1 if its page is not there.
__device__ __forceinline__ int64_t cache_row(const KvLaunch &p, int b, int kh, int t) {
  uint32_t pg, off;
  p.page.split((uint32_t)t, pg, off);
  const int64_t page = p.a.table ? p.a.table[(int64_t)b * p.a.table_pages + pg] : b;
  if (page < 0 || page >= p.a.cache.pages) return -1;
  return (page * p.a.cache.heads + kh) * p.a.cache.page + off;
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

// A scale byte as attention reads it: 253 and more are NaN.
__device__ __forceinline__ bool kv_nan(uint32_t s) { return s >= 253; }
__device__ __forceinline__ float kv_scale(uint32_t s) { return mx_scale(kv_nan(s) ? 255 : s); }

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

hipError_t launch_kv_rows(const KvLaunch &p, int64_t tiles);

}  // namespace oq
