// vq_fp8_device.h -- e4m3 quantization of 128-column blocks, shared by the
// quantizer and the norms.
#pragma once

#include "vq_device.h"

namespace vqmi {

constexpr int kFp8Block = 128;       // columns (and weight rows) that share a scale
constexpr float kFp8Max = 448.0f;    // largest e4m3 value
constexpr uint32_t kFp8Nan = 0x7fu;

// Two fp32 values as fp16 (or bf16) bits, rounded to nearest even.
__device__ __forceinline__ uint32_t pack16(float a, float b, bool f16) {
  if (f16) return __builtin_bit_cast(uint32_t, half2_t{(_Float16)a, (_Float16)b});
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float float2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(float2_t{a, b}, bf16x2));
}

// Maximum over the 16 lanes of a DPP row, in every lane of it (rotations by
// 1, 2, 4 and 8).
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
#define VQMI_ROR(ctrl) (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, true)
  v = max(v, VQMI_ROR(0x121));
  v = max(v, VQMI_ROR(0x122));
  v = max(v, VQMI_ROR(0x124));
  v = max(v, VQMI_ROR(0x128));
#undef VQMI_ROR
  return v;
}

// The scale of a block whose largest finite magnitude is amax: amax / 448
// rounded to nearest, or 1 where that is 0 (a block of zeros, or of values up
// to 3e-43, which the e4m3 codes of x / 1 take as zeros too).
__device__ __forceinline__ float fp8_scale(float amax) {
  const float s = __fdiv_rn(amax, kFp8Max);
  return s > 0.0f ? s : 1.0f;
}

// x / s on its way to the nearest e4m3 value: the fp32 quotient with its last
// bit set where it is not exact ("rounded to odd"), so that the conversion's
// round-to-nearest-even sees which side of a tie the true quotient lies on.
// rs is about 1 / s; both are normal numbers.
__device__ __forceinline__ float fp8_quotient(float x, float s, float rs) {
  const float a = fabsf(x);
  float q = a * rs;
  q = fmaf(fmaf(-q, s, a), rs, q);   // within a unit of the quotient
  const float r = fmaf(-q, s, a);    // exact; +0 where q is the quotient
  uint32_t u = __float_as_uint(q) + (uint32_t)((int32_t)__float_as_uint(r) >> 31);  // at or below the quotient
  u |= r != 0.0f ? 1u : 0u;
  return __uint_as_float((u & 0x7fffffffu) | (__float_as_uint(x) & 0x80000000u));
}

__device__ __forceinline__ u32x2 fp8_convert8(const float* q) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return u32x2{(uint32_t)lo, (uint32_t)hi};
}

// Blocks with NaN or infinities (NaN codes, which do not count for the scale),
// and blocks so small that 1 / s overflows or s loses bits (lifted by 2^64
// first, quotients cut at 448).  Called by whole waves.
__device__ __forceinline__ u32x2 fp8_quantize8_odd(const float* x, float* scale) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.0f);
  amax = __uint_as_float(row16_max(__float_as_uint(amax)));
  const float s = fp8_scale(amax), lift = amax < 0x1p-60f ? 0x1p64f : 1.0f;
  const float sl = s * lift, rs = 1.0f / sl;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf(fp8_quotient(x[i] * lift, sl, rs), -kFp8Max), kFp8Max);
  const u32x2 c = fp8_convert8(q);
  uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t sh = 8u * (i & 3);
    if (!(fabsf(x[i]) < INFINITY)) w[i >> 2] = (w[i >> 2] & ~(0xffu << sh)) | (kFp8Nan << sh);
  }
  *scale = s;
  return u32x2{w[0], w[1]};
}

// Eight values of a block of 128 that 16 neighbouring lanes hold, to e4m3
// codes; `top`: the largest magnitude of the lane's eight, as fp32 bits (NaN
// above infinity).  Called by whole waves.
__device__ __forceinline__ u32x2 fp8_quantize8(const float* x, uint32_t top, float* scale) {
  top = row16_max(top);
  const bool odd = top >= 0x7f800000u || (top != 0u && top < 0x21800000u);  // not finite, or below 2^-60
  if (__ballot(odd) != 0ull) return fp8_quantize8_odd(x, scale);
  const float s = fp8_scale(__uint_as_float(top)), rs = 1.0f / s;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = fp8_quotient(x[i], s, rs);
  *scale = s;
  return fp8_convert8(q);
}

// The largest magnitude of eight values, as fp32 bits.
__device__ __forceinline__ uint32_t abs_max8(const float* x) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  return m;
}

}  // namespace vqmi
