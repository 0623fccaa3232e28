// vq_mx4_device.h -- tensors of 4-bit e2m1 values with a power-of-two scale for
// each 32 columns: how a wave loads them and multiplies them, shared by the
// product and the mixture-of-experts layer.
//
// A wave's operands.  Lane l stands for row (or token) l % 16 of 16 and holds,
// for each step of 128 * PCS columns, PCS whole blocks of 32 columns: blocks
// PCS * (l / 16) to PCS * (l / 16) + PCS - 1 of the step.  So its values are
// 16 * PCS consecutive bytes and its scales PCS consecutive bytes, which the
// matrix instructions take byte by byte from one register; both operands are
// laid out the same way, so columns meet their own.
//
// Two kinds of products.
//   4-bit x 4-bit: one 16 x 16 x 128 instruction per block of a lane, with
//   both scales applied inside.  Products of two e2m1 values are whole
//   quarters of at most 36, so the 32 of a block sum exactly; the blocks and the accumulator join as fp32
//   does: measured over every spread of the scales, an instruction is off by
//   at most 4 units of 2^-24 of the largest block sum or accumulator (its
//   products are not cut the way the e4m3 instructions cut theirs).
//   4-bit x 16-bit: the 4-bit values times their scale are bf16 values, and
//   fp16 values where the scale is between 2^-23 and 2^13, so one conversion
//   per pair feeds the 16 x 16 x 32 instructions, whose products are exact.
//   With fp16 activations, steps that hold another scale take x apart into two
//   bf16 values instead (11 bits are 8 and 3), and twice the instructions.
#pragma once

#include "vq_block_device.h"
#include "vq_block_kernels.h"

#include <type_traits>

namespace vqmi {

typedef int int8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kMx4Block = 32;  // columns that share a scale

constexpr int kMx4Planes = 3;  // fp32 as a sum of three bf16 planes

// acc + the product of 16 rows and 16 tokens over a block of every lane, whose
// scales are bytes J of sa and sb.
template <int J>
__device__ __forceinline__ float4_t mx4_mfma(u32x4 a, u32x4 b, float4_t acc, uint32_t sa, uint32_t sb) {
  const int8v av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const int8v bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc, 4, 4, J, (int)sa, J, (int)sb);
}

// Eight codes times 2^(scale - 127) as bf16 or fp16 (scale: the byte in an fp32
// exponent's place; 255 gives NaN).
__device__ __forceinline__ bf16x8_t mx4_bf16(uint32_t codes, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
__device__ __forceinline__ half8_t mx4_half(uint32_t codes, float scale) {
  const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 0);
  const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 1);
  const half2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 2);
  const half2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 3);
  return half8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Byte J of `scales` as the fp32 number with that exponent.
template <int J>
__device__ __forceinline__ float mx4_scale(uint32_t scales) {
  return __uint_as_float((J < 3 ? scales >> (8 * J) & 0xffu : scales >> 24) << 23);
}

// The PCS scale bytes within [104, 140] (2^-23 to 2^13), where e2m1 values times
// the scale are fp16 values.
template <int PCS>
__device__ __forceinline__ bool mx4_scales_fit_half(uint32_t s) {
  bool ok = true;
#pragma unroll
  for (int j = 0; j < PCS; ++j) ok = ok && (s >> (8 * j) & 0xffu) - 104u <= 36u;
  return ok;
}

// PCS blocks of a lane: codes and scale bytes.  Blocks past the last column (or
// a row past the last: `row` is kOutOfRange) arrive as zeros with a scale of 1.
template <int PCS>
struct Mx4Frag {
  u32x4 q[PCS];
  uint32_t s;
};
// Row `row` of buffers with `pitch` blocks a row, blocks from `block` on that
// come before `end`; whole: scales a row and `end` are multiples of PCS, and the
// scales lie on a multiple of PCS bytes.
template <int PCS>
__device__ __forceinline__ void mx4_load(Mx4Frag<PCS>& f, rsrc_t qr, rsrc_t sr, uint32_t row, uint32_t block,
                                         uint32_t end, uint32_t pitch, bool whole) {
  const bool live = row != kOutOfRange;
  const uint32_t at = row * pitch + block;
#pragma unroll
  for (int j = 0; j < PCS; ++j) f.q[j] = buf_load_b128(qr, live && block + j < end ? (at + j) * 16u : kOutOfRange);
  if (whole) {  // then `end` is a multiple of PCS: a lane's blocks are all there or none is
    const bool in = live && block < end;
    const uint32_t off = in ? at : kOutOfRange;
    uint32_t s;
    if constexpr (PCS == 4) s = buf_load_b32(sr, off);
    else if constexpr (PCS == 2) s = buf_load_b16(sr, off);
    else s = __builtin_amdgcn_raw_buffer_load_b8(sr, off, 0, 0);
    f.s = in ? s : 0x7f7f7f7fu;
  } else {
    f.s = 0u;
#pragma unroll
    for (int j = 0; j < PCS; ++j) {
      const bool in = live && block + j < end;
      const uint32_t s = __builtin_amdgcn_raw_buffer_load_b8(sr, in ? at + j : kOutOfRange, 0, 0);
      f.s |= (in ? s : 0x7fu) << (8 * j);
    }
  }
}

// A lane's 32 * PCS values of 16-bit activations, PLANES of them; `row`: the
// byte offset of the token's row (kOutOfRange: zeros).
template <int PCS, int PLANES>
struct Mx4XFrag {
  u32x4 v[PLANES][PCS][4];
};
template <int PCS, int PLANES>
__device__ __forceinline__ void mx4_load_x(Mx4XFrag<PCS, PLANES>& f, rsrc_t xr, uint32_t row, uint32_t plane_bytes,
                                           uint32_t block, uint32_t end) {
#pragma unroll
  for (int p = 0; p < PLANES; ++p) {
#pragma unroll
    for (int j = 0; j < PCS; ++j) {
      const uint32_t off = block + j < end && row != kOutOfRange ? row + p * plane_bytes + (block + j) * 64u : kOutOfRange;
#pragma unroll
      for (int i = 0; i < 4; ++i) f.v[p][j][i] = buf_load_b128(xr, off + (off == kOutOfRange ? 0u : 16u * i));
    }
  }
}

// Eight fp16 values as two bf16 parts whose sum they are.
__device__ __forceinline__ void mx4_split_half(u32x4 x, bf16x8_t* hi, bf16x8_t* lo) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const half2_t v = __builtin_bit_cast(half2_t, w[i]);
    const float f[2] = {(float)v.x, (float)v.y};
    uint32_t a[2], b[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      a[k] = __float_as_uint(f[k]) & 0xffff0000u;  // a NaN's quiet bit is among these
      const float r = f[k] - __uint_as_float(a[k]);
      b[k] = fabsf(f[k]) < INFINITY ? __float_as_uint(r) : 0u;
    }
    h[i] = a[0] >> 16 | a[1];
    l[i] = b[0] >> 16 | (b[1] & 0xffff0000u);
  }
  *hi = __builtin_bit_cast(bf16x8_t, u32x4{h[0], h[1], h[2], h[3]});
  *lo = __builtin_bit_cast(bf16x8_t, u32x4{l[0], l[1], l[2], l[3]});
}

// acc[n] += 16 rows times 16 tokens of tile n over block J of every lane.
template <int XK, int J, int NT, int PCS, int PLANES>
__device__ __forceinline__ void mx4_dot16(const Mx4Frag<PCS>& w, const Mx4XFrag<PCS, PLANES>* x, float4_t* acc,
                                          bool fit_half) {
  const float s = mx4_scale<J>(w.s);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (XK == kMx4XF16) {
      if (fit_half) {
        const half8_t a = mx4_half(w.q[J][i], s);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, __builtin_bit_cast(half8_t, x[n].v[0][J][i]), acc[n], 0, 0, 0);
      } else {
        const bf16x8_t a = mx4_bf16(w.q[J][i], s);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          bf16x8_t hi, lo;
          mx4_split_half(x[n].v[0][J][i], &hi, &lo);
          acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, lo, acc[n], 0, 0, 0);
          acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, hi, acc[n], 0, 0, 0);
        }
      }
    } else {
      const bf16x8_t a = mx4_bf16(w.q[J][i], s);
#pragma unroll
      for (int p = PLANES - 1; p >= 0; --p) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, x[n].v[p][J][i]), acc[n], 0, 0, 0);
      }
    }
  }
}

// The same over all of a lane's blocks.
template <int XK, int NT, int PCS, int PLANES>
__device__ __forceinline__ void mx4_dot16s(const Mx4Frag<PCS>& w, const Mx4XFrag<PCS, PLANES>* x, float4_t* acc,
                                           bool fit_half) {
  mx4_dot16<XK, 0, NT>(w, x, acc, fit_half);
  if constexpr (PCS > 1) mx4_dot16<XK, 1, NT>(w, x, acc, fit_half);
  if constexpr (PCS > 2) {
    mx4_dot16<XK, 2, NT>(w, x, acc, fit_half);
    mx4_dot16<XK, 3, NT>(w, x, acc, fit_half);
  }
}

// A step's operands: 16 rows of w and NT tiles of 16 tokens.
template <int XK, int PCS, int NT>
struct Mx4Step {
  typedef std::conditional_t<XK == kMx4XMx4, Mx4Frag<PCS>, Mx4XFrag<PCS, 1>> X;
  Mx4Frag<PCS> w;
  X x[NT];

  __device__ __forceinline__ void dot(float4_t* acc) const {
    if constexpr (XK == kMx4XMx4) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        acc[n] = mx4_mfma<0>(w.q[0], x[n].q[0], acc[n], w.s, x[n].s);
        if constexpr (PCS > 1) acc[n] = mx4_mfma<1>(w.q[1], x[n].q[1], acc[n], w.s, x[n].s);
        if constexpr (PCS > 2) {
          acc[n] = mx4_mfma<2>(w.q[2], x[n].q[2], acc[n], w.s, x[n].s);
          acc[n] = mx4_mfma<3>(w.q[3], x[n].q[3], acc[n], w.s, x[n].s);
        }
      }
    } else {
      mx4_dot16s<XK, NT>(w, x, acc, XK == kMx4XF16 && __ballot(!mx4_scales_fit_half<PCS>(w.s)) == 0ull);
    }
  }
};

}  // namespace vqmi
