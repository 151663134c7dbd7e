// mx.hip -- microscaled (MX) quantization and its read-back.
//
// A block of 32 consecutive elements of a row shares one power of two
// 2^(s - 127), stored as the byte s.  With m = max |x| over the block and
// E(m) its biased fp32 exponent, s = max(E(m) - e_max, 0): the exponent of
// the largest element lands on the largest exponent of the element type
// (e_max = 2 for e2m1, 8 for e4m3).  An element is x / 2^(s - 127) rounded
// to nearest even in its type, at most the type's largest value.  Division
// by a power of two is exact, so the codes are a function of the input
// alone; there is no accumulated error to bound.
//
// Memory bound: one pass, 16 bytes of bf16 a lane.  Measured beside a large
// copy's 5.3 TB/s: 13824 x 5120 bf16 to e2m1 36 us (5.0 TB/s), fp32 to e2m1 66 us
// (4.9), e2m1 to bf16 26 us (the codes come from the Infinity Cache); 32760 x
// 5120 bf16 to e4m3 83 to 105 us by what ran before it (6.1 to 4.8), fp32 to
// e4m3 180 us (4.7), e4m3 to bf16 83 us (6.1), to fp32 205 us (4.1).  The
// smallest calls are a launch (1.8 to 2.8 us).
#include <hip/hip_runtime.h>

#include "mx_codec.h"
#include "oq_internal.h"

namespace oq {
namespace {

// One thread takes 8 elements, four neighbouring lanes a block.
template <class T, int FMT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const T *__restrict__ x, int64_t chunks,
                                                          uint8_t *__restrict__ codes,
                                                          uint8_t *__restrict__ scales) {
  for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < chunks;
       c += (int64_t)gridDim.x * 256) {
    float v[8];
    load8(x + 8 * c, v);
    mx_store8<FMT>(v, c, codes, scales);
  }
}

template <class T, int FMT>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales,
                                                            int64_t chunks, T *__restrict__ out) {
  for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < chunks;
       c += (int64_t)gridDim.x * 256) {
    float v[8];
    mx_load8<FMT>(codes, scales, c, v);
    store8(out + 8 * c, v);
  }
}

unsigned grid_for(int64_t chunks) {
  const int64_t g = (chunks + 255) / 256;
  return (unsigned)(g < 16384 ? g : 16384);
}

}  // namespace

hipError_t launch_mx_quantize(const void *x, int dtype, int64_t rows, int d, int format,
                              uint8_t *codes, uint8_t *scales, hipStream_t stream) {
  const int64_t chunks = rows * (d / 8);
  const dim3 g(grid_for(chunks)), b(256);
#define OQ_CASE(DT, T, F)                                                                    \
  if (dtype == DT && format == F)                                                            \
    hipLaunchKernelGGL((mx_quantize_kernel<T, F>), g, b, 0, stream, (const T *)x, chunks, codes, \
                       scales);
  OQ_CASE(0, float, 0) OQ_CASE(0, float, 1) OQ_CASE(1, uint16_t, 0) OQ_CASE(1, uint16_t, 1)
#undef OQ_CASE
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int format,
                                int64_t rows, int d, int dtype, void *out, hipStream_t stream) {
  const int64_t chunks = rows * (d / 8);
  const dim3 g(grid_for(chunks)), b(256);
#define OQ_CASE(DT, T, F)                                                                       \
  if (dtype == DT && format == F)                                                               \
    hipLaunchKernelGGL((mx_dequantize_kernel<T, F>), g, b, 0, stream, codes, scales, chunks, (T *)out);
  OQ_CASE(0, float, 0) OQ_CASE(0, float, 1) OQ_CASE(1, uint16_t, 0) OQ_CASE(1, uint16_t, 1)
#undef OQ_CASE
  return hipGetLastError();
}

}  // namespace oq
