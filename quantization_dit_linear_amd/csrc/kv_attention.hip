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

// A row's parts, in their order: four elements a thread.
template <class T>
__global__ __launch_bounds__(256) void kv_join_kernel(KvLaunch p) {
  const KvAttentionArgs &a = p.a;
  const KvTile t = find_tile(p, blockIdx.x);
  if (t.b < 0) return;
  const int hd = a.cache.head_dim, q4 = hd / 4;
  const int64_t total = a.q_tokens * a.q_heads;
  const int rows = t.rows - t.row0 < p.rows ? t.rows - t.row0 : p.rows;
  for (int e = threadIdx.x; e < rows * q4; e += 256) {
    uint32_t i, h;
    const int r = e / q4, d = 4 * (e - r * q4);
    p.share.split((uint32_t)(t.row0 + r), i, h);
    const int64_t tok = t.start + (int64_t)i, head = (int64_t)blockIdx.y * p.share.d + h;
    const int64_t row = tok * a.q_heads + head;
    float top = -kInf, sum = 0.f;
    for (int s = 0; s < p.splits; s++) top = fmaxf(top, p.part_ml[s * total + row][0]);
    const float base = top == -kInf ? 0.f : top;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < p.splits; s++) {
      const f32x2 ml = p.part_ml[s * total + row];
      if (ml[1] == 0.f) continue;  // a part that saw nothing left no sum
      const float f = __builtin_amdgcn_exp2f(ml[0] - base);
      sum += ml[1] * f;
      v += *(const f32x4 *)(p.part + (s * total + row) * hd + d) * f;
    }
    if (sum == 0.f) v = f32x4{0.f, 0.f, 0.f, 0.f};
    else v *= 1.f / sum;
    store4((T *)a.out + tok * a.out_token + head * a.out_head + d, v);
    if (a.lse && d == 0) a.lse[row] = lse_of(top, sum);
  }
}

// The launch that the sizes decide: rows of a tile, tiles, parts.
struct Plan {
  int rows, splits;
  int64_t tiles;
};

Plan plan(int dtype, int64_t q_tokens, int q_heads, int kv_heads, int head_dim, int64_t batch, int64_t capacity) {
  const int64_t share = q_heads / kv_heads, per = q_tokens * share / batch;  // rows of a sequence, on average
  Plan r;
  r.rows = dtype == 0 || per <= 16 ? 16 : 32;
  // every sequence may end inside a tile
  r.tiles = (q_tokens * share + r.rows - 1) / r.rows + batch;
  const int64_t groups = ((per + r.rows - 1) / r.rows) * batch * kv_heads;
  // parts of at least 256 tokens, until four workgroups a CU are there
  int64_t s = (1024 + groups - 1) / std::max<int64_t>(1, groups);
  s = std::min({s, (capacity + 255) / 256, (int64_t)128});
  r.splits = (int)std::max<int64_t>(1, s);
  return r;
}

}  // namespace

int64_t kv_attention_workspace(int64_t q_tokens, int q_heads, int kv_heads, int head_dim,
                               int64_t batch, int64_t capacity) {
  int64_t most = 0;  // for either type
  for (int dtype = 0; dtype < 2; dtype++) {
    const Plan r = plan(dtype, q_tokens, q_heads, kv_heads, head_dim, batch, capacity);
    if (r.splits > 1) most = std::max(most, (int64_t)r.splits * q_tokens * q_heads * (head_dim + 2) * 4);
  }
  return most;
}

hipError_t launch_kv_attention(const KvAttentionArgs &a) {
  const Plan r = plan(a.dtype, a.q_tokens, a.q_heads, a.cache.heads, a.cache.head_dim, a.batch,
                      (int64_t)a.table_pages * a.cache.page);
  const int64_t share = a.q_heads / a.cache.heads, n = a.q_starts ? 0 : a.q_tokens / a.batch;
  const int64_t each = std::max<int64_t>(1, (n * share + r.rows - 1) / r.rows);
  const int64_t tiles = a.q_starts ? r.tiles : each * a.batch, total = a.q_tokens * a.q_heads;
  KvLaunch p{a, FastDiv((uint32_t)a.cache.page), FastDiv((uint32_t)share), FastDiv((uint32_t)each), r.rows,
             r.splits, fabsf(a.scale) * 1.4426950408889634f, nullptr, nullptr};
  // hidden tokens are scores of -infinity, which a factor of 0 would make NaN: the
  // smallest number instead, by which every finite score is as good as 0
  if (p.log2_scale == 0.f) p.log2_scale = std::numeric_limits<float>::denorm_min();
  p.part = (float *)a.workspace;
  p.part_ml = (f32x2 *)(p.part + r.splits * total * a.cache.head_dim);
  hipError_t e = launch_kv_rows(p, tiles);
  if (e != hipSuccess || r.splits == 1) return e;
  const dim3 grid((unsigned)tiles, (unsigned)a.cache.heads);
  if (a.dtype == 0) hipLaunchKernelGGL((kv_join_kernel<float>), grid, dim3(256), 0, a.stream, p);
  else hipLaunchKernelGGL((kv_join_kernel<uint16_t>), grid, dim3(256), 0, a.stream, p);
  return hipGetLastError();
}

}  // namespace oq
