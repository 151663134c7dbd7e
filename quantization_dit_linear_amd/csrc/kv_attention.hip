// kv_attention.hip -- attention of new queries over the 4-bit key/value cache:
// which kernel takes a call, in how many parts, and the join of the parts.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c q k_j - m),  lse = (m + log2 sum_j p_j) ln 2
// with c = scale log2 e and m the running maximum of a row's c q k_j.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <limits>
#include <stdlib.h>

#include "kv_attention.h"

namespace oq {
namespace {

// A group's parts, in their order.  A workgroup takes every gridDim.z-th row of a
// group; 256 / (head_dim / 4) threads an element take every so many parts, eight
// loads at a time, and their sums join in a fixed order.
constexpr int kMaxWorkers = 2048;

template <class T>
__global__ __launch_bounds__(256) void kv_join_kernel(KvLaunch p) {
  __shared__ __attribute__((aligned(16))) float sums[256 * 4];
  __shared__ float weight[kMaxWorkers], part_sum[4], part_top[4];
  const KvAttentionArgs &a = p.a;
  const int tid = threadIdx.x, hd = a.cache.head_dim, q4 = hd / 4, groups = 256 / q4;
  const KvTile t = find_tile(p, blockIdx.x);
  if (t.b < 0) return;
  const int2 which = p.parts[(int64_t)blockIdx.x * a.cache.heads + blockIdx.y];
  const int first = which.x, parts = which.y;
  if (parts == 1) return;
  // part k: the last of its worker where the group starts there, else the first
  const auto slot = [&](int k) { return (int64_t)(k == 0 ? first : first - 1 + 2 * k) * p.rows; };
  const int rows = t.rows - t.row0 < p.rows ? t.rows - t.row0 : p.rows;
  for (int r = blockIdx.z; r < rows; r += gridDim.z) {
    __syncthreads();  // the row before is read
    float top = -kInf, sum = 0.f;
    for (int k = tid; k < parts; k += 256) top = fmaxf(top, p.part_ml[slot(k) + r][0]);
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    if ((tid & 63) == 0) part_top[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(part_top[0], part_top[1]), fmaxf(part_top[2], part_top[3]));
    const float base = top == -kInf ? 0.f : top;
    for (int k = tid; k < parts; k += 256) {
      const f32x2 ml = p.part_ml[slot(k) + r];
      const float w = __builtin_amdgcn_exp2f(ml[0] - base);
      sum += ml[1] * w;
      weight[k] = ml[1] == 0.f ? -1.f : w;  // a part that saw nothing left no sum: it is not read
    }
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    if ((tid & 63) == 0) part_sum[tid >> 6] = sum;
    __syncthreads();
    sum = part_sum[0] + part_sum[1] + part_sum[2] + part_sum[3];

    const int g = tid / q4, d = 4 * (tid - g * q4);
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (g < groups) {
      for (int k0 = g; k0 < parts; k0 += 8 * groups) {
        f32x4 x[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int k = k0 + e * groups;
          x[e] = f32x4{0.f, 0.f, 0.f, 0.f};
          if (k < parts && weight[k] != -1.f) x[e] = *(const f32x4 *)(p.part + (slot(k) + r) * hd + d) * weight[k];
        }
#pragma unroll
        for (int e = 0; e < 8; e++) v += x[e];
      }
      *(f32x4 *)(sums + 4 * tid) = v;
    }
    __syncthreads();
    if (g == 0) {
      for (int k = 1; k < groups; k++) v += *(const f32x4 *)(sums + 4 * (tid + k * q4));
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

// The launch that the sizes decide.
struct Plan {
  int rows, step, workers;
  int64_t tiles;
  int64_t workspace(int kv_heads, int head_dim) const {
    return workers ? (int64_t)2 * workers * rows * (head_dim + 2) * 4 + tiles * kv_heads * 8 : 0;
  }
};

Plan plan(int dtype, int64_t q_tokens, int q_heads, int kv_heads, int head_dim, int64_t batch, int64_t capacity) {
  const int64_t share = q_heads / kv_heads, per = q_tokens * share / batch;  // rows of a sequence, on average
  Plan r;
  r.rows = dtype == 0 || head_dim > 128 || per <= 16 ? 16 : 32;
  r.step = kv_rows_step(head_dim);
  // every sequence may end inside a tile
  r.tiles = (q_tokens * share + r.rows - 1) / r.rows + batch;
  const char *e2 = getenv("KV_WG"), *e3 = getenv("KV_MAX");
  const int64_t most = e3 ? atoi(e3) : 1024;
  const int64_t units = r.tiles * kv_heads * (capacity / r.step + 8);
  r.workers = r.tiles <= most && units < (int64_t)1 << 30 ? (e2 ? atoi(e2) : 2048) : 0;
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
  const char *e1 = getenv("KV_LEAST"), *e2 = getenv("KV_EXTRA");
  KvLaunch p{a, FastDiv((uint32_t)a.cache.page), FastDiv((uint32_t)share), FastDiv((uint32_t)each), r.rows,
             r.step, e2 ? atoi(e2) : 2, (int)tiles, r.workers, e1 ? atoi(e1) : 2, fabsf(a.scale) * 1.4426950408889634f, nullptr, nullptr, nullptr};
  // hidden tokens are scores of -infinity, which a factor of 0 would make NaN: the
  // smallest number instead, by which every finite score is as good as 0
  if (p.log2_scale == 0.f) p.log2_scale = std::numeric_limits<float>::denorm_min();
  p.part = (float *)a.workspace;
  p.part_ml = (f32x2 *)(p.part + (int64_t)2 * r.workers * r.rows * a.cache.head_dim);
  p.parts = (int2 *)(p.part_ml + (int64_t)2 * r.workers * r.rows);
  hipError_t e = launch_kv_rows(p);
  if (e != hipSuccess || !r.workers) return e;
  // a workgroup a row where the groups are few
  const dim3 grid((unsigned)tiles, (unsigned)a.cache.heads, tiles * a.cache.heads <= 128 ? r.rows : 1);
  if (a.dtype == 0) hipLaunchKernelGGL((kv_join_kernel<float>), grid, dim3(256), 0, a.stream, p);
  else hipLaunchKernelGGL((kv_join_kernel<uint16_t>), grid, dim3(256), 0, a.stream, p);
  return hipGetLastError();
}

}  // namespace oq
