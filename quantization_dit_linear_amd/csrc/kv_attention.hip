// kv_attention.hip -- attention of new queries over the 4-bit key/value cache:
// which kernel takes a call, in how many parts, and the join of the parts.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c q k_j - m),  lse = (m + log2 sum_j p_j) ln 2
// with c = scale log2 e and m the running maximum of a row's c q k_j.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <limits>

#include "kv_attention.h"

namespace oq {
namespace {

// Whether a group has parts to join.  (Starts that descend leave what the workspace
// held before: nothing beyond it is read.)
__device__ __forceinline__ bool joins(const KvLaunch &p, int first, int parts) {
  return parts > 1 && parts <= p.workers + 1 && first >= 0 && first < 2 * p.workers && first - 1 + 2 * (parts - 1) < 2 * p.workers;
}

// A group's parts, in their order, a wave a row: 64 parts' maxima and sums of
// weights a time, then their sums, as many side by side as the lanes hold, eight
// loads a lane.  SPLIT: the waves of a workgroup share a row (parts are many where
// groups are few), and the first of them adds up.
template <class T, bool SPLIT>
__global__ __launch_bounds__(SPLIT ? 1024 : 256) void kv_join_kernel(KvLaunch p) {
  constexpr int kWaves = SPLIT ? 16 : 4;
  __shared__ __attribute__((aligned(16))) float sums[kWaves][64 * 4];
  __shared__ f32x2 waves[kWaves];
  const KvAttentionArgs &a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hd = a.cache.head_dim, q4 = hd / 4, side = 64 / q4, g = lane / q4, d = 4 * (lane - g * q4);
  const int2 which = p.parts[(int64_t)blockIdx.x * a.cache.heads + blockIdx.y];
  const KvTile t = find_tile(p, blockIdx.x);
  if (t.b < 0) return;
  const int first = which.x, parts = which.y;
  if (!joins(p, first, parts)) return;
  // part k: the last of its worker where the group starts there, else the first
  const auto slot = [&](int k) { return (int64_t)(k == 0 ? first : first - 1 + 2 * k) * p.rows; };
  const int rows = t.rows - t.row0 < p.rows ? t.rows - t.row0 : p.rows;
  const int per = SPLIT ? (parts + kWaves - 1) / kWaves : parts;
  const int k0 = SPLIT ? wave * per : 0, k1 = k0 + per < parts ? k0 + per : parts;
  for (int r = SPLIT ? blockIdx.z : blockIdx.z * kWaves + wave; r < rows; r += SPLIT ? gridDim.z : kWaves * gridDim.z) {
    float top = -kInf, sum = 0.f;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int c0 = k0; c0 < k1; c0 += 64) {
      const int k = c0 + lane, n = k1 - c0 < 64 ? k1 - c0 : 64;
      f32x2 ml = {-kInf, 0.f};
      if (k < k1) ml = p.part_ml[slot(k) + r];
      float now = ml[0];
      for (int off = 32; off > 0; off >>= 1) now = fmaxf(now, __shfl_xor(now, off));
      now = fmaxf(now, top);
      const float base = now == -kInf ? 0.f : now, old = __builtin_amdgcn_exp2f(top - base);
      const float w = __builtin_amdgcn_exp2f(ml[0] - base);
      top = now;
      v *= old;
      float s = ml[1] * w;
      for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
      sum = sum * old + s;
      const float keep = ml[1] == 0.f ? -1.f : w;  // a part that saw nothing left no sum: it is not read
      for (int b0 = 0; b0 < n; b0 += 8 * side) {
        f32x4 x[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int at = b0 + e * side + g;
          const float f = __shfl(keep, at & 63);
          x[e] = f32x4{0.f, 0.f, 0.f, 0.f};
          if (g < side && at < n && f != -1.f) x[e] = *(const f32x4 *)(p.part + (slot(c0 + at) + r) * hd + d) * f;
        }
#pragma unroll
        for (int e = 0; e < 8; e++) v += x[e];
      }
    }
    // lanes exchange their sums, without SPLIT within the wave: the hardware keeps its LDS
    // operations in their order, the fence keeps the compiler to it
    const auto turn = [] {
      if (SPLIT) __syncthreads();
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    };
    turn();  // the row before is read
    *(f32x4 *)&sums[wave][4 * lane] = v;
    if (lane == 0) waves[wave] = f32x2{top, sum};
    turn();
    if (SPLIT && wave != 0) continue;
    if (lane < q4) {
      v = f32x4{0.f, 0.f, 0.f, 0.f};
      if (SPLIT) {
#pragma unroll
        for (int w = 0; w < kWaves; w++) top = fmaxf(top, waves[w][0]);
        sum = 0.f;
      }
      const float base = top == -kInf ? 0.f : top;
      for (int w = SPLIT ? 0 : wave; w <= (SPLIT ? kWaves - 1 : wave); w++) {
        const float f = SPLIT ? __builtin_amdgcn_exp2f(waves[w][0] - base) : 1.f;
        if (SPLIT) sum += waves[w][1] * f;
        for (int k = 0; k < side; k++) v += *(const f32x4 *)&sums[w][4 * (lane + k * q4)] * f;
      }
      if (sum == 0.f) v = f32x4{0.f, 0.f, 0.f, 0.f};
      else v *= 1.f / sum;
      uint32_t i, h;
      p.share.split((uint32_t)(t.row0 + r), i, h);
      const int64_t tok = t.start + (int64_t)i, head = (int64_t)blockIdx.y * p.share.d + h;
      store4((T *)a.out + tok * a.out_token + head * a.out_head + d, v);
      if (a.lse && d == 0) a.lse[tok * a.q_heads + head] = lse_of(top, sum);
    }
  }
}

// The same for tiles of many rows, whose parts are few: four elements a thread.
template <class T>
__global__ __launch_bounds__(256) void kv_join_wide_kernel(KvLaunch p) {
  const KvAttentionArgs &a = p.a;
  const int2 which = p.parts[(int64_t)blockIdx.x * a.cache.heads + blockIdx.y];
  const KvTile t = find_tile(p, blockIdx.x);
  if (t.b < 0) return;
  const int first = which.x, parts = which.y, hd = a.cache.head_dim, q4 = hd / 4;
  const int e = (int)blockIdx.z * 256 + (int)threadIdx.x, r = e / q4, d = 4 * (e - r * q4);
  if (!joins(p, first, parts) || r >= p.rows || t.row0 + r >= t.rows) return;
  const auto slot = [&](int k) { return (int64_t)(k == 0 ? first : first - 1 + 2 * k) * p.rows + r; };
  float top = -kInf, sum = 0.f;
  for (int k = 0; k < parts; k++) top = fmaxf(top, p.part_ml[slot(k)][0]);
  const float base = top == -kInf ? 0.f : top;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int k = 0; k < parts; k++) {
    const f32x2 ml = p.part_ml[slot(k)];
    if (ml[1] == 0.f) continue;  // a part that saw nothing left no sum
    const float w = __builtin_amdgcn_exp2f(ml[0] - base);
    sum += ml[1] * w;
    v += *(const f32x4 *)(p.part + slot(k) * hd + d) * w;
  }
  if (sum == 0.f) v = f32x4{0.f, 0.f, 0.f, 0.f};
  else v *= 1.f / sum;
  uint32_t i, h;
  p.share.split((uint32_t)(t.row0 + r), i, h);
  const int64_t tok = t.start + (int64_t)i, head = (int64_t)blockIdx.y * p.share.d + h;
  store4((T *)a.out + tok * a.out_token + head * a.out_head + d, v);
  if (a.lse && d == 0) a.lse[tok * a.q_heads + head] = lse_of(top, sum);
}

// Rows of a sequence, on average, from which on the tiles kernel takes a call, rows
// against tiles kernel: 64 sequences of 2048 tokens, 8 heads of 4 queries, 64 rows 81
// against 137 us, 128 rows 142 against 142; 8 of 4096 tokens 46 against 49 and 65
// against 53 us; one of 32760 tokens 47 against 67 and 71 against 70 us; 6 of 2040
// tokens with heads of 64 in fp32 54 against 27 us and 32 against 30.
// One kernel takes the whole call: 63 single tokens (over up to 8192) beside a prompt of
// 4096, 32 query and 8 key heads, 555 us, as two calls 56 and 254 us.
constexpr int kWide = 64;

// Groups (a tile of rows and a head) up to which their many parts are joined by the
// waves of a workgroup together and their steps taken by teams of waves (fewer parts):
// 48 groups 37 against 57 us with a wave a row, 128 groups 70 against 41 us.
constexpr int kFew = 64;

// The launch that the sizes decide.
struct Plan {
  int rows, step, workers;
  bool team, wide;  // wide: the tiles kernel
  int64_t tiles;
  int64_t workspace(int kv_heads, int head_dim) const {
    return workers ? (int64_t)2 * workers * rows * (head_dim + 2) * 4 + tiles * kv_heads * 8 : 0;
  }
};

Plan plan(int dtype, int64_t q_tokens, int q_heads, int kv_heads, int head_dim, int64_t batch, int64_t capacity) {
  const int64_t share = q_heads / kv_heads, per = q_tokens * share / batch;  // rows of a sequence, on average
  Plan r;
  r.wide = per > kWide;
  r.rows = r.wide ? kv_tiles_rows(dtype, head_dim) : 16;
  r.step = r.wide ? kKvTilesStep : kv_rows_step(head_dim);
  // every sequence may end inside a tile
  r.tiles = (q_tokens * share + r.rows - 1) / r.rows + batch;
  // Even shares of the steps while the tiles are few enough to be counted by every
  // wave: eight waves a CU, or two workgroups of them where the groups are so few that
  // each is cut into many parts (fewer parts to join: one token over 32760 24.3
  // against 26 us).  Beyond 1024 tiles a wave takes a group.  One token of each of n
  // sequences, 8 query heads a key head, shared out against a wave a group: n = 256 up to
  // 4096 tokens, one key head, 36 against 92 us, up to 512 tokens 24 against 18; n = 1100
  // 52 against 23 us (up to 512) and 104 against 121 us (up to 4096), with 8 key heads 170
  // against 96 and 570 against 531; n = 4000 197 against 43 and 399 against 262 us.  What
  // it does not even out: one of 32768 among 1099 of up to 512 tokens, 90 against 652 us.
  const int64_t units = r.tiles * kv_heads * (capacity / r.step + 8);
  r.workers = r.tiles <= 1024 && units < (int64_t)1 << 30 ? 2048 : 0;
  r.team = r.workers && r.tiles * kv_heads <= kFew;
  if (r.team) r.workers /= 4;
  // The tiles kernel up to 1024 groups, four a CU: 1560 x 32760, 40 heads (280) 1150
  // against 1950 us; a causal prompt of 2048 tokens, 8 key heads of 4 (264) 80 against 73,
  // of 4096 (520) 255 against 247, of 8192 (1032) 948 against 728 us, all tokens seen 1057
  // against 1046.
  if (r.wide) r.team = false, r.workers = r.workers && r.tiles * kv_heads <= 1024 ? 256 : 0;
  return r;
}

}  // namespace

int64_t kv_attention_workspace(int64_t q_tokens, int q_heads, int kv_heads, int head_dim,
                               int64_t batch, int64_t capacity) {
  int64_t most = 0;  // for either type
  for (int dtype = 0; dtype < 2; dtype++)
    most = std::max(most, plan(dtype, q_tokens, q_heads, kv_heads, head_dim, batch, capacity).workspace(kv_heads, head_dim));
  return most;
}

hipError_t launch_kv_attention(const KvAttentionArgs &a) {
  const Plan r = plan(a.dtype, a.q_tokens, a.q_heads, a.cache.heads, a.cache.head_dim, a.batch,
                      (int64_t)a.table_pages * a.cache.page);
  const int64_t share = a.q_heads / a.cache.heads, n = a.q_starts ? 0 : a.q_tokens / a.batch;
  const int64_t each = std::max<int64_t>(1, (n * share + r.rows - 1) / r.rows);
  const int64_t tiles = a.q_starts ? r.tiles : each * a.batch;
  KvLaunch p{a, FastDiv((uint32_t)a.cache.page), FastDiv((uint32_t)share), FastDiv((uint32_t)each), r.rows,
             r.step, 2, (int)tiles, r.workers, 2, (int)n, r.team, fabsf(a.scale) * 1.4426950408889634f, nullptr, nullptr, nullptr};
  // hidden tokens are scores of -infinity, which a factor of 0 would make NaN: the
  // smallest number instead, by which every finite score is as good as 0
  if (p.log2_scale == 0.f) p.log2_scale = std::numeric_limits<float>::denorm_min();
  p.part = (float *)a.workspace;
  p.part_ml = (f32x2 *)(p.part + (int64_t)2 * r.workers * r.rows * a.cache.head_dim);
  p.parts = (int2 *)(p.part_ml + (int64_t)2 * r.workers * r.rows);
  hipError_t e = r.wide ? launch_kv_tiles(p) : launch_kv_rows(p);
  if (e != hipSuccess || !r.workers) return e;
  if (r.wide) {
    const dim3 grid((unsigned)tiles, (unsigned)a.cache.heads, (unsigned)(r.rows * a.cache.head_dim / 4 + 255) / 256);
    if (a.dtype == 0) hipLaunchKernelGGL((kv_join_wide_kernel<float>), grid, dim3(256), 0, a.stream, p);
    else hipLaunchKernelGGL((kv_join_wide_kernel<uint16_t>), grid, dim3(256), 0, a.stream, p);
    return hipGetLastError();
  }
  // a workgroup a row where the groups are few
  const bool few = tiles * a.cache.heads <= kFew;
  const dim3 grid((unsigned)tiles, (unsigned)a.cache.heads, few ? r.rows : 1);
  if (a.dtype == 0) {
    if (few) hipLaunchKernelGGL((kv_join_kernel<float, true>), grid, dim3(1024), 0, a.stream, p);
    else hipLaunchKernelGGL((kv_join_kernel<float, false>), grid, dim3(256), 0, a.stream, p);
  } else {
    if (few) hipLaunchKernelGGL((kv_join_kernel<uint16_t, true>), grid, dim3(1024), 0, a.stream, p);
    else hipLaunchKernelGGL((kv_join_kernel<uint16_t, false>), grid, dim3(256), 0, a.stream, p);
  }
  return hipGetLastError();
}

}  // namespace oq
