// oq_internal.h -- definitions shared by the host side of liborbitquant and
// its HIP kernels (not part of the public ABI).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace oq {

// Raise a kernel's dynamic-LDS limit on the current device, once per device
// (`done` holds one bit per device id; setting the attribute twice from two
// threads is harmless).
inline hipError_t ensure_lds_limit(const void *fn, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (uint64_t)1 << dev : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return hipSuccess;
  e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  if (bit) done.fetch_or(bit, std::memory_order_release);
  return hipSuccess;
}

constexpr int kMaxD = 16384;
constexpr int kGroup = 128;  // coordinates per storage-order group
// token lengths d: multiples of kDimStep (a last partial group of 32, 64 or
// 96 coordinates is stored in coordinate order); linear K: multiples of the
// linear's 64-slot K step
constexpr int kDimStep = 32;
constexpr int kLinearKStep = 64;

// Slot size of the bf16 fast rotate kernel for token size d: the Hadamard
// block, at most 1024 coordinates (a block of 2048 or 4096 spans several
// slots), 512 at d = 5120 and 3072 (a batch of two tokens then tiles the
// kernel's compute waves).  The host lays out the kernel's LDS copy of a
// token by slots, so both sides take the size from here.
constexpr __host__ __device__ int fast_slot(int d) {
  const int h = d & -d, cap = (d == 5120 || d == 3072) ? 512 : 1024;
  return h < cap ? h : cap;
}

// Unit-variance decision thresholds of one codebook (fp32, ascending).
struct Thresholds {
  float t[15];
  int count;  // 2^bits - 1
};

// Unit-variance levels of one codebook, as fp16 bit patterns.
struct LevelsF16 {
  uint16_t v[16];
};

// Unit-variance levels of one codebook, fp32 (dequantized outputs).
struct LevelsF32 {
  float v[16];
};

// Device-side rotation plan for one (device, d, seed).
struct DevicePlan {
  int d = 0, h = 0;
  // scatter table for the generic kernel: entry j = pi^-1(j), bit 31 set when
  // the sign applied at that destination is negative.
  int32_t *scatter = nullptr;         // with signs
  int32_t *scatter_nosign = nullptr;  // signs dropped
  // tables of the bf16 fast path: byte offset 2 pi^-1(j) of every source
  // element j inside a token's LDS copy, and per source dword the XOR mask
  // that applies the destination's sign to both bf16 halves.
  uint32_t *fast_scatter = nullptr;
  uint32_t *fast_signs = nullptr;
  uint32_t *fast_nosigns = nullptr;
  // input already in rotation order (x'_i = x_{pi(i)}): identity placement
  int32_t *scatter_id = nullptr;   // generic kernel: j | sign bit of D_j
  uint32_t *fast_signs_id = nullptr;  // fast path: per dword pair, signs of D_j, D_j+1
  int32_t *perm_inv = nullptr;     // pi^-1 (row permutation of oq_permute_rows)
  int pins = 0;  // explicit handles (oq_plan_create) holding this plan
};

struct RotateArgs {
  const void *x;
  int dtype;  // 0 fp32, 1 bf16
  int64_t n_tok;
  int d, h, bits;
  bool signs;
  bool rotated_out;  // fp32 rotated unit vector instead of codes
  bool dequant_out;  // bf16 s * level[code] instead of codes
  bool input_permuted;  // x already in rotation order: D and H only
  LevelsF32 levels;  // unit levels (dequant_out)
  void *out;
  float *norms;
  hipStream_t stream;
};

// Kernel launchers (defined in the .hip files).  Return a hipError_t.
// General kernel.  Up to 4 bits the codebook comes in th and a.levels; at 8
// bits from the device table (layout above).
hipError_t launch_rotate_quantize_generic(const RotateArgs &a, const DevicePlan &p,
                                          const Thresholds &th, const uint32_t *table);
// bf16 fast path; sets *handled = false (and does nothing) for shapes it does
// not cover.  table: the device codebook table of a.bits (layout above).
hipError_t launch_rotate_quantize_fast(const RotateArgs &a, const uint32_t *scat,
                                       const uint32_t *smask, const uint32_t *table,
                                       bool *handled);
// Device codebook table of one (bits, family, d): the fast path's cell grid
// ({tau, base} per cell), then the 2^bits unit levels (fp32), then the
// 2^bits - 1 unit thresholds (fp32), all as 32-bit words.  The grid is 1/8
// of a unit over [-130, 130) up to 4 bits -- every sqrt(d) z of a unit
// vector with d <= 16384 lies inside, so a kernel needs no clamp -- and
// 1/128 over [-5, 5) at 8 bits.
constexpr int kFastHalfUnits = 130;
constexpr int kFastCells = 16 * kFastHalfUnits;
constexpr int kFastCells8 = 1280;
constexpr __host__ __device__ int cells_for_bits(int bits) {
  return bits == 8 ? kFastCells8 : kFastCells;
}
constexpr __host__ __device__ int table_levels_word(int bits) { return 2 * cells_for_bits(bits); }
constexpr __host__ __device__ int table_thresholds_word(int bits) {
  return 2 * cells_for_bits(bits) + (1 << bits);
}

struct LinearArgs {
  const uint8_t *a_codes;
  const float *a_norms;
  int a_bits;
  const uint8_t *w_codes;
  const float *w_norms;
  int w_bits;
  int64_t M, N;
  int K;
  uint16_t *y;
  hipStream_t stream;
};

// Up to 4 bits the levels come as fp16 bit patterns in la / lw; at 8 bits
// as the fp32 unit levels of the device tables ta / tw (layout above).
hipError_t launch_linear(const LinearArgs &a, const LevelsF16 &la, const LevelsF16 &lw,
                         const uint32_t *ta, const uint32_t *tw);

// INT4 weight-only round-to-nearest (AdaLN projections)
hipError_t launch_rtn4_prepare(const void *W, int dtype, int64_t rows, int d, uint8_t *q4,
                               float *scales, hipStream_t stream);
hipError_t launch_rtn4_linear(const void *x, int dtype, int64_t M, const uint8_t *q4,
                              const float *scales, int64_t N, int K, uint16_t *y,
                              hipStream_t stream);

// dst row pi^-1(j) = src row j, i.e. dst[i] = src[pi(i)], rows of row_bytes
hipError_t launch_permute_rows(const void *src, void *dst, int64_t rows, int64_t row_bytes,
                               const int32_t *perm_inv, hipStream_t stream);

// Microscaled (MX) codes: format 0 = e2m1 (4 bits), 1 = e4m3 (8 bits), blocks
// of kMxBlock elements with a power-of-two scale byte.
constexpr int kMxBlock = 32;
hipError_t launch_mx_quantize(const void *x, int dtype, int64_t rows, int d, int format,
                              uint8_t *codes, uint8_t *scales, hipStream_t stream);
hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int format,
                                int64_t rows, int d, int dtype, void *out, hipStream_t stream);

struct MxLinearArgs {
  const uint8_t *a_codes, *a_scales;
  int a_format;
  const uint8_t *w_codes, *w_scales;
  int w_format;
  int64_t M, N;
  int K;
  uint16_t *y;
  hipStream_t stream;
};
hipError_t launch_mx_linear(const MxLinearArgs &a);

struct RmsNormArgs {
  const void *x, *residual;
  int dtype;
  int64_t rows;
  int d;
  float eps;
  const void *weight, *gate, *scale, *shift;  // any may be null
  int param_dtype;
  int64_t rows_per_mod, mod_stride;
  void *sum;  // may be null
  int out;    // 0: y in dtype, 1: MX e4m3, 2: MX e2m1
  void *y;
  uint8_t *y_scales;
  hipStream_t stream;
};
hipError_t launch_rms_norm(const RmsNormArgs &a);

constexpr int kRopeMaxHeadDim = 512, kRopeMaxAxes = 4;
struct RopeArgs {
  const void *x;
  int dtype;
  int64_t tokens;
  int heads, head_dim, turned;  // turned: leading elements of a head that are paired
  int64_t x_token, x_head, y_token, y_head;  // strides in elements
  const int32_t *pos;                        // [tokens][axes]
  int axes;
  bool half, inverse;
  void *y;
  hipStream_t stream;
  uint64_t freq[kRopeMaxHeadDim / 2];  // turns per position of each pair, units of 2^-64
  uint8_t axis[kRopeMaxHeadDim / 2];   // the axis of each pair
};
hipError_t launch_rope(const RopeArgs &a);

// INT4 weights with group scales and, where zeros is not null, zero points
hipError_t launch_rtn4_group_prepare(const void *W, int dtype, int64_t rows, int d, int group,
                                     uint8_t *q4, void *scales, void *zeros, int scale_dtype,
                                     hipStream_t stream);
struct Rtn4GroupArgs {
  const void *x;
  int dtype;
  int64_t M;
  const uint8_t *q4;
  const void *scales, *zeros;  // zeros may be null
  int scale_dtype, group;
  int64_t N;
  int K;
  uint16_t *y;
  hipStream_t stream;
};
hipError_t launch_rtn4_group_linear(const Rtn4GroupArgs &a);

struct QkNormRopeArgs {
  struct Side {  // queries or keys
    const void *x;
    void *y;
    const void *weight;  // may be null
    int64_t x_token, x_head, y_token, y_head;
    int heads;
  } side[2];
  int dtype, param_dtype;
  int64_t tokens;
  int head_dim, turned;
  float eps;
  const int32_t *pos;
  int axes;
  bool half;
  hipStream_t stream;
  uint64_t freq[kRopeMaxHeadDim / 2];
  uint8_t axis[kRopeMaxHeadDim / 2];
};
hipError_t launch_qk_norm_rope(const QkNormRopeArgs &a);

// The 4-bit key/value cache: [pages][heads][page][head_dim / 2] codes and
// [pages][heads][page][head_dim / 32] scale bytes.
constexpr int kKvMaxHeadDim = 256, kKvMaxHeads = 65535;
constexpr int64_t kKvMaxRows = (int64_t)1 << 27, kKvMaxBatch = (int64_t)1 << 20,
                  kKvMaxLength = (int64_t)1 << 30;
struct KvCache {
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int64_t pages;
  int heads, page, head_dim;
};
struct KvWriteArgs {
  const void *k, *v;
  int dtype;
  int64_t tokens, k_token, k_head, v_token, v_head;
  const int64_t *slots;
  KvCache cache;
  hipStream_t stream;
};
hipError_t launch_kv_write(const KvWriteArgs &a);

struct KvAttentionArgs {
  const void *q;
  int dtype;
  int64_t q_tokens, q_token, q_head;
  int q_heads;
  KvCache cache;
  int batch;
  const int32_t *lengths, *q_starts, *table;  // q_starts and table may be null
  int table_pages;
  float scale;
  bool causal;
  int window;
  void *out;
  int64_t out_token, out_head;
  float *lse;  // may be null
  void *workspace;
  hipStream_t stream;
};
int64_t kv_attention_workspace(int64_t q_tokens, int q_heads, int kv_heads, int head_dim,
                               int64_t batch, int64_t capacity);
hipError_t launch_kv_attention(const KvAttentionArgs &a);

}  // namespace oq
