// kv_cache.hip -- keys and values of new tokens into the 4-bit cache.
//
// Each head's row is quantized as mx.hip does (blocks of 32, e2m1 elements with
// a power-of-two scale) and stored at its token's slot.  Memory bound: 16 or 32
// bytes of input a lane, four lanes a block; a token's heads lie a page of rows
// apart in the cache, so the stores are pieces of head_dim / 2 bytes.  4680 tokens of
// 40 + 40 heads of 128, bf16 (121 MB): 22.4 us, 5.4 TB/s.
#include <hip/hip_runtime.h>

#include "kv_cache.h"
#include "mx_codec.h"
#include "oq_internal.h"

namespace oq {
namespace {

// A workgroup takes `group` tokens of the keys (blockIdx.y 0) or values; item i
// is 8 elements: chunk i % chunks of head i / chunks % heads of a token.
template <class T>
__global__ __launch_bounds__(256) void kv_write_kernel(KvWriteArgs a, int group, FastDiv chunks,
                                                       FastDiv row_chunks) {
  const bool second = blockIdx.y != 0;
  const T *x = (const T *)(second ? a.v : a.k);
  const int64_t x_token = second ? a.v_token : a.k_token, x_head = second ? a.v_head : a.k_head;
  uint8_t *codes = second ? a.cache.v_codes : a.cache.k_codes;
  uint8_t *scales = second ? a.cache.v_scales : a.cache.k_scales;
  const int64_t slots = a.cache.pages * a.cache.page;
  for (int64_t t0 = (int64_t)blockIdx.x * group; t0 < a.tokens; t0 += (int64_t)gridDim.x * group) {
    const int nt = a.tokens - t0 < group ? (int)(a.tokens - t0) : group;
    for (uint32_t i = threadIdx.x; i < nt * row_chunks.d; i += 256) {
      uint32_t t, w, h, c;
      row_chunks.split(i, t, w);
      chunks.split(w, h, c);
      const int64_t slot = a.slots[t0 + t];
      if (slot < 0 || slot >= slots) continue;  // the four lanes of a block agree
      float v[8];
      load8(x + (t0 + t) * x_token + h * x_head + 8 * c, v);
      // (in 64 bits: a cache may have more slots than 2^32)
      const int64_t p = slot / a.cache.page, r = slot - p * a.cache.page;
      mx_store8<0>(v, ((p * a.cache.heads + h) * a.cache.page + r) * chunks.d + c, codes, scales);
    }
  }
}

}  // namespace

hipError_t launch_kv_write(const KvWriteArgs &a) {
  const int chunks = a.cache.head_dim / 8;
  const int64_t row = (int64_t)chunks * a.cache.heads;
  int64_t group = 1024 / row;  // about four items a thread, where tokens are short
  if (group < 1 || a.tokens < 1024 * group) group = 1;
  const int64_t gx = (a.tokens + group - 1) / group;
  const dim3 grid((unsigned)(gx < (1 << 20) ? gx : 1 << 20), 2);
  const FastDiv c((uint32_t)chunks), r((uint32_t)row);
  if (a.dtype == 0)
    hipLaunchKernelGGL((kv_write_kernel<float>), grid, dim3(256), 0, a.stream, a, (int)group, c, r);
  else
    hipLaunchKernelGGL((kv_write_kernel<uint16_t>), grid, dim3(256), 0, a.stream, a, (int)group, c, r);
  return hipGetLastError();
}

}  // namespace oq
