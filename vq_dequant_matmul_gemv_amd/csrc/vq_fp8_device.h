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
__device__ __forceinline__ float row16_max(float v) {
#define VQMI_ROR_MAX(ctrl) \
  v = fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, 0xf, 0xf, true)))
  VQMI_ROR_MAX(0x121);
  VQMI_ROR_MAX(0x122);
  VQMI_ROR_MAX(0x124);
  VQMI_ROR_MAX(0x128);
#undef VQMI_ROR_MAX
  return v;
}

// The scale of a block whose largest finite magnitude is amax: amax / 448
// rounded to nearest (1 for a block of zeros).
__device__ __forceinline__ float fp8_scale(float amax) { return amax > 0.0f ? __fdiv_rn(amax, kFp8Max) : 1.0f; }

// x / s on its way to the nearest e4m3 value: the fp32 quotient with its last
// bit set where it is not exact ("rounded to odd"), so that the conversion's
// round-to-nearest-even sees which side of a tie the true quotient lies on.
// x and s come premultiplied by the same power of two, so s and 1 / s are
// normal; rs is about 1 / s.
__device__ __forceinline__ float fp8_quotient(float x, float s, float rs) {
  const float a = fabsf(x);
  float q = a * rs;
  q = fmaf(fmaf(-q, s, a), rs, q);        // within half a unit of the quotient, but for rare last bits
  const float r = fmaf(-q, s, a);         // exact
  uint32_t u = __float_as_uint(q);
  u = r < 0.0f ? u - 1u : u;              // now at or below the true quotient
  u |= r != 0.0f ? 1u : 0u;
  q = fminf(__uint_as_float(u), kFp8Max);
  return copysignf(q, x);
}

// Power of two that lifts a block of tiny values (and its scale) into the
// range where 1 / s is finite; 1 for every other block.
__device__ __forceinline__ float fp8_lift(float amax) { return amax < 0x1p-60f ? 0x1p64f : 1.0f; }

// Eight values of a block (any finite or not) to e4m3 codes, given the
// block's scale and lift.  NaN and infinities become NaN codes.
__device__ __forceinline__ u32x2 fp8_pack8(const float* x, float s, float lift) {
  const float sl = s * lift, rs = 1.0f / sl;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = fp8_quotient(x[i] * lift, sl, rs);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], v, true);
    w[h] = (uint32_t)v;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t sh = 8u * (i & 3);
    if (!(fabsf(x[i]) < INFINITY)) w[i >> 2] = (w[i >> 2] & ~(0xffu << sh)) | (kFp8Nan << sh);
  }
  return u32x2{w[0], w[1]};
}

__device__ __forceinline__ float finite_abs(float v) { const float a = fabsf(v); return a < INFINITY ? a : 0.0f; }

}  // namespace vqmi
