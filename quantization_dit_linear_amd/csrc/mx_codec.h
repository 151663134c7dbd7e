// mx_codec.h -- device helpers shared by the kernels that read or write
// microscaled (MX) codes and 8-element pieces of fp32 or bf16 rows.
//
// T = float is fp32, T = uint16_t holds bf16 bit patterns; FMT 0 is e2m1
// (two codes a byte, the even element in the low half), 1 is e4m3.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace oq {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void unpack8(const u32x4 &w, float *v) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
  }
}

// bf16 rounding is the hardware's round to nearest even
__device__ __forceinline__ u32x4 pack8(const float *v) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const bf16x2 p = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
    w[i] = __builtin_bit_cast(uint32_t, p);
  }
  return w;
}

__device__ __forceinline__ void load8(const uint16_t *p, float *v) { unpack8(*(const u32x4 *)p, v); }

__device__ __forceinline__ void load8(const float *p, float *v) {
  const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = a[i], v[4 + i] = b[i];
}

__device__ __forceinline__ void store8(uint16_t *p, const float *v) { *(u32x4 *)p = pack8(v); }

__device__ __forceinline__ void store8(float *p, const float *v) {
  *(f32x4 *)p = f32x4{v[0], v[1], v[2], v[3]};
  *(f32x4 *)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}

// 16 bytes of a row: 8 bf16 or 4 fp32 elements
__device__ __forceinline__ void load16(const uint16_t *p, float *v) { load8(p, v); }

__device__ __forceinline__ void load16(const float *p, float *v) {
  const f32x4 a = *(const f32x4 *)p;
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = a[i];
}

// stores of rows that the kernel does not read again: non-temporal, so that
// they do not push what is still to be read out of the caches
__device__ __forceinline__ void store8_nt(uint16_t *p, const float *v) {
  __builtin_nontemporal_store(pack8(v), (u32x4 *)p);
}

__device__ __forceinline__ void store8_nt(float *p, const float *v) {
  __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, (f32x4 *)p);
  __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, (f32x4 *)(p + 4));
}

__device__ __forceinline__ void store16_nt(uint16_t *p, const float *v) { store8_nt(p, v); }

__device__ __forceinline__ void store16_nt(float *p, const float *v) {
  __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, (f32x4 *)p);
}

// 2^(s - 127) of a scale byte; 255 stands for a block that held a NaN or an
// infinity and reads back as NaN.
__device__ __forceinline__ float mx_scale(uint32_t s) {
  const uint32_t b = s == 0 ? 1u << 22 : s == 255 ? 0x7fc00000u : s << 23;
  return __builtin_bit_cast(float, b);
}

// max over the four lanes of a block (lanes 4i .. 4i+3): DPP quad exchanges
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  uint32_t o = __builtin_amdgcn_update_dpp(0, m, 0xB1, 0xf, 0xf, true);  // lanes 1,0,3,2
  m = m > o ? m : o;
  o = __builtin_amdgcn_update_dpp(0, m, 0x4E, 0xf, 0xf, true);  // lanes 2,3,0,1
  return m > o ? m : o;
}

// Quantizes 8 elements, chunk c of a matrix whose rows are whole blocks, and
// stores their codes; four neighbouring lanes hold a block's chunks (all of
// them active) and one of them stores its scale byte.  The maximum is taken
// over the absolute bit patterns, which order like the values and put NaN
// above infinity above every number.
template <int FMT>
__device__ __forceinline__ void mx_store8(const float *v, int64_t c, uint8_t *codes,
                                          uint8_t *scales) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
    m = m > b ? m : b;
  }
  m = quad_max(m);
  constexpr int EMAX = FMT == 0 ? 2 : 8;
  const int e = (int)(m >> 23);
  const bool bad = e == 255;
  const uint32_t s = bad ? 255u : e > EMAX ? (uint32_t)(e - EMAX) : 0u;
  const float sc = __builtin_bit_cast(float, bad ? 0x7f000000u : s == 0 ? 1u << 22 : s << 23);
  if constexpr (FMT == 0) {
    uint32_t w = 0;  // the hardware's conversion rounds to nearest even and saturates at 6
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], sc, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], sc, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], sc, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], sc, 3);
    *(uint32_t *)(codes + 4 * c) = bad ? 0u : w;
  } else {
    // the hardware's e4m3 conversion turns values above 464 into NaN: clamp
    // to 448 first (the block's largest value can be anything below 512)
    const float top = 448.f * sc;
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; i++) t[i] = __builtin_amdgcn_fmed3f(v[i], -top, top);
    i16x2 a = {0, 0}, b = {0, 0};
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, t[0], t[1], sc, false);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, t[2], t[3], sc, true);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, t[4], t[5], sc, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, t[6], t[7], sc, true);
    u32x2 w = {__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
    if (bad) w = u32x2{0u, 0u};
    *(u32x2 *)(codes + 8 * c) = w;
  }
  if ((c & 3) == 0) scales[c >> 2] = (uint8_t)s;
}

// The 8 values of chunk c.  Elements are decoded at unit scale and
// multiplied by the block's power of two in fp32: exact (also as bf16, whose
// smallest subnormal lies below 2^-128), and NaN where the scale is.
template <int FMT>
__device__ __forceinline__ void mx_load8(const uint8_t *codes, const uint8_t *scales, int64_t c,
                                         float *v) {
  const float sc = mx_scale(scales[c >> 2]);
  f32x2 p[4];
  if constexpr (FMT == 0) {
    const uint32_t w = *(const uint32_t *)(codes + 4 * c);
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  } else {
    const u32x2 w = *(const u32x2 *)(codes + 8 * c);
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[0], 1.0f, false);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[0], 1.0f, true);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[1], 1.0f, false);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[1], 1.0f, true);
  }
#pragma unroll
  for (int i = 0; i < 4; i++) v[2 * i] = p[i][0] * sc, v[2 * i + 1] = p[i][1] * sc;
}

}  // namespace oq
