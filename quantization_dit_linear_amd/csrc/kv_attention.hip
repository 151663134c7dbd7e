// kv_attention.hip -- attention of new queries over the 4-bit key/value cache.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q k_j - m),  lse = m + ln sum_j p_j
// in one pass over the tokens with a running maximum m.
#include <hip/hip_runtime.h>

#include "kv_cache.h"
#include "mx_codec.h"
#include "oq_internal.h"

namespace oq {
namespace {

constexpr float kInf = __builtin_huge_valf();

// A scale byte as attention reads it: 253 and more are NaN.
__device__ __forceinline__ float kv_scale(uint32_t s) { return mx_scale(s >= 253 ? 255 : s); }

__device__ __forceinline__ float fp4(uint32_t nibble) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(nibble, 1.0f, 0)[0];
}

// One wave a query head: 64 tokens a step, a token a lane for the scores, an
// element a lane for the sum.
template <class T>
__global__ __launch_bounds__(64) void kv_attention_kernel(KvAttentionArgs a, FastDiv page) {
  __shared__ float qs[kKvMaxHeadDim], ps[64];
  __shared__ int64_t rows[64];
  const KvCache &c = a.cache;
  const int lane = threadIdx.x, hd = c.head_dim, nb = hd / 32, share = a.q_heads / c.heads;
  const int64_t cap = (int64_t)a.table_pages * c.page;
  for (int64_t r = blockIdx.x; r < a.q_tokens * a.q_heads; r += gridDim.x) {
    const int64_t tok = r / a.q_heads;
    const int h = (int)(r - tok * a.q_heads), kh = h / share;
    // the sequence: the last whose start is not behind the token
    int b, i, n;
    if (a.q_starts) {
      int lo = 0, hi = a.batch;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (a.q_starts[mid] <= tok) lo = mid + 1;
        else hi = mid;
      }
      b = lo - 1;
      if (b < 0 || tok >= a.q_starts[b + 1]) continue;
      i = (int)(tok - a.q_starts[b]), n = a.q_starts[b + 1] - a.q_starts[b];
    } else {
      n = (int)(a.q_tokens / a.batch);
      b = (int)(tok / n), i = (int)(tok - (int64_t)b * n);
    }
    int64_t len = a.lengths[b];
    len = len < 0 ? 0 : len > cap ? cap : len;
    const int64_t at = len - n + i;
    int64_t hi = a.causal && at + 1 < len ? at + 1 : len, lo = a.window && at + 1 > a.window ? at + 1 - a.window : 0;
    const T *q = (const T *)a.q + tok * a.q_token + h * a.q_head;
    __syncthreads();
    for (int e = lane; e < hd; e += 64) {
      if constexpr (sizeof(T) == 2) qs[e] = __builtin_bit_cast(float, (uint32_t)q[e] << 16);
      else qs[e] = q[e];
    }
    float m = -kInf, l = 0.f, acc[kKvMaxHeadDim / 64] = {};
    for (int64_t t0 = lo; t0 < hi; t0 += 64) {
      __syncthreads();
      const int64_t t = t0 + lane;
      float s = -kInf;
      if (t < hi) {
        uint32_t p, off;
        page.split((uint32_t)t, p, off);
        const int64_t pg = a.table ? a.table[(int64_t)b * a.table_pages + p] : b;
        const bool bad = pg < 0 || pg >= c.pages;
        const int64_t row = ((bad ? 0 : pg) * c.heads + kh) * c.page + off;
        rows[lane] = row;
        s = bad ? __builtin_nanf("") : 0.f;
        for (int k = 0; k < nb; k++) {
          float u = 0.f;
          for (int e = 0; e < 16; e++) {
            const uint32_t w = c.k_codes[row * (hd / 2) + 16 * k + e];
            u = fmaf(qs[32 * k + 2 * e], fp4(w & 15), u);
            u = fmaf(qs[32 * k + 2 * e + 1], fp4(w >> 4), u);
          }
          s = fmaf(u, kv_scale(c.k_scales[row * nb + k]), s);
        }
        s *= a.scale;
      }
      float top = s;
      for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
      top = fmaxf(m, top);
      const float base = top == -kInf ? 0.f : top, old = expf(m - base);
      const float p = t < hi ? expf(s - base) : 0.f;
      m = top;
      float sum = p;
      for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
      l = fmaf(l, old, sum);
      ps[lane] = p;
      __syncthreads();
      for (int x = 0; x < kKvMaxHeadDim / 64; x++) {
        const int e = lane + 64 * x;
        if (e >= hd) break;
        float o = acc[x] * old;
        for (int j = 0; j < 64 && t0 + j < hi; j++) {
          const uint32_t w = c.v_codes[rows[j] * (hd / 2) + e / 2];
          o = fmaf(ps[j], fp4(w >> (4 * (e & 1)) & 15) * kv_scale(c.v_scales[rows[j] * nb + e / 32]), o);
        }
        acc[x] = o;
      }
    }
    T *out = (T *)a.out + tok * a.out_token + h * a.out_head;
    for (int x = 0; x < kKvMaxHeadDim / 64; x++) {
      const int e = lane + 64 * x;
      if (e >= hd) break;
      const float o = l == 0.f ? 0.f : acc[x] / l;
      if constexpr (sizeof(T) == 2) out[e] = __builtin_bit_cast(uint16_t, (__bf16)o);
      else out[e] = o;
    }
    if (a.lse && lane == 0) a.lse[r] = l == 0.f ? -kInf : m + logf(l);
  }
}

}  // namespace

int64_t kv_attention_workspace(int64_t q_tokens, int q_heads, int kv_heads, int head_dim,
                               int64_t batch, int64_t capacity) {
  return 0;
}

hipError_t launch_kv_attention(const KvAttentionArgs &a) {
  const int64_t rows = a.q_tokens * a.q_heads;
  const dim3 grid((unsigned)(rows < (1 << 20) ? rows : 1 << 20));
  const FastDiv page((uint32_t)a.cache.page);
  if (a.dtype == 0)
    hipLaunchKernelGGL((kv_attention_kernel<float>), grid, dim3(64), 0, a.stream, a, page);
  else
    hipLaunchKernelGGL((kv_attention_kernel<uint16_t>), grid, dim3(64), 0, a.stream, a, page);
  return hipGetLastError();
}

}  // namespace oq
