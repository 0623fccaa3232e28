// vq_mx4_device.h -- tensors of 4-bit e2m1 values with a power-of-two scale for
// each 32 columns: how a wave loads them and multiplies them, shared by the
// product and the mixture-of-experts layer.
//
// A wave's operands.  Lane l stands for row (or token) l % 16 of 16 and holds,
// for each step of 256 columns, blocks 2 * (l / 16) and 2 * (l / 16) + 1 of the
// step's eight: 32 consecutive bytes of values and two of scales, which the
// matrix instructions take byte by byte from one register.  Both operands are
// laid out the same way, so columns meet their own.
//
// Memory holds rows side by side, and a wave that reads 16 bytes of 16 rows at
// once moves a quarter of what whole lines would: so values are loaded a row's
// 128 bytes by 8 lanes and change places in LDS, in a slot that only the wave
// itself uses (no barriers; LDS runs a wave's accesses in order).
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

// Both scale bytes within [104, 140] (2^-23 to 2^13), where e2m1 values times
// the scale are fp16 values.
__device__ __forceinline__ bool mx4_scales_fit_half(uint32_t s) {
  return (s & 0xffu) - 104u <= 36u && (s >> 8 & 0xffu) - 104u <= 36u;
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

// Eight of a row's values times eight of a token's, over a step's four lane
// groups: 16 rows x 16 tokens x 32 columns.  x: 16-bit values, or (bf16) the
// planes whose sum they are.
template <int XK>
__device__ __forceinline__ float4_t mx4_mfma16(uint32_t codes, float scale, u32x4 x, float4_t acc, bool fit_half) {
  if constexpr (XK == kMx4XF16) {
    if (fit_half)
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(mx4_half(codes, scale), __builtin_bit_cast(half8_t, x), acc, 0, 0, 0);
    const bf16x8_t a = mx4_bf16(codes, scale);
    bf16x8_t hi, lo;
    mx4_split_half(x, &hi, &lo);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, lo, acc, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, hi, acc, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx4_bf16(codes, scale), __builtin_bit_cast(bf16x8_t, x), acc, 0, 0, 0);
  }
}

// ---------------------------------------------------------------------------
// a wave's stream over the columns: 16 rows of w, up to 16 rows of activations
//
// XK: what the activations are; PL: planes of them; NL: load instructions for a
// step's rows of a plane (8 rows each of 4-bit values, 2 of 16-bit ones);
// DEPTH: steps in flight.
// ---------------------------------------------------------------------------
template <int XK, int PL, int NL>
struct Mx4Slot {
  static constexpr int kRows = NL * (XK == kMx4XMx4 ? 8 : 2);  // rows of activations
  u32x4 w[16 * 8];
  u32x4 x[PL][NL * 64];
  uint32_t ws[16 * 4], xs[XK == kMx4XMx4 ? 16 * 4 : 1];  // scales: the words they lie in
};

// The row a lane loads for: of w's values by instruction i, of scales, and of
// the activations by instruction i.
__device__ __forceinline__ int mx4_w_row(int i, int lane) { return 8 * i + (lane >> 3); }
__device__ __forceinline__ int mx4_s_row(int lane) { return lane >> 2; }
template <int XK>
__device__ __forceinline__ int mx4_x_row(int i, int lane) {
  return XK == kMx4XMx4 ? 8 * i + (lane >> 3) : 2 * i + (lane >> 5);
}

// Rows of scales, which may start at any byte: a step's eight lie in three
// aligned words at most, the first of them `skew` bytes before the row's.  No
// word without a byte of the tensor's is read.
struct Mx4Scales {
  rsrc_t rsrc;
  uint32_t base_skew;
  __device__ __forceinline__ Mx4Scales(const uint8_t* base, uint32_t bytes)
      : rsrc(make_rsrc(base - (reinterpret_cast<uintptr_t>(base) & 3u),
                       ((reinterpret_cast<uintptr_t>(base) & 3u) + (uint64_t)bytes + 3) & ~(uint64_t)3)),
        base_skew((uint32_t)reinterpret_cast<uintptr_t>(base) & 3u) {}
  // The lane's word of scales from byte `at` of the tensor on.
  __device__ __forceinline__ uint32_t word(uint32_t at, int lane) const {
    return (lane & 3) < 3 ? ((base_skew + at) & ~3u) + 4 * (lane & 3) : kOutOfRange;
  }
  __device__ __forceinline__ uint32_t skew(uint32_t at) const { return (base_skew + at) & 3u; }
};

// What a wave loads its steps from: 16 rows of w and rows of activations.
template <int NL>
struct Mx4Source {
  rsrc_t wr, wsr;               // values and scales of the rows
  uint32_t wsoff, xoff[NL];     // byte offsets of the lane's rows; kOutOfRange: no such row
  uint32_t ws_skew;             // of the row that the lane multiplies

  __device__ __forceinline__ void take(const Mx4Source& o) {
    wr = o.wr, wsr = o.wsr, wsoff = o.wsoff, ws_skew = o.ws_skew;
#pragma unroll
    for (int i = 0; i < NL; ++i) xoff[i] = o.xoff[i];
  }
};

template <int XK, int PL, int NL, int DEPTH>
struct Mx4Stream {
  typedef Mx4Slot<XK, PL, NL> Slot;
  typedef Mx4Source<NL> Source;
  static constexpr uint32_t kXBlock = XK == kMx4XMx4 ? 16 : 64;  // bytes of a block of activations
  rsrc_t xr, xsr;
  uint32_t woff[2], xsoff, xs_skew;
  uint32_t plane;       // bytes from one plane of activations to the next
  uint32_t first, end;  // blocks of columns: the first one, and behind the last
  int column;           // the row of activations that the lane multiplies
  Slot* slot;
  u32x4 w[DEPTH][2], x[DEPTH][PL][NL];
  uint32_t ws[DEPTH], xs[DEPTH];

  __device__ __forceinline__ void load(int j, const Source& src, uint32_t k, int lane) {  // step k; past the end: zeros
    const uint32_t b = first + k * 8;
    const bool in_w = b + (lane & 7) < end;
#pragma unroll
    for (int i = 0; i < 2; ++i) w[j][i] = buf_load_b128(src.wr, in_w ? woff[i] + b * 16 + (lane & 7) * 16 : kOutOfRange);
    ws[j] = buf_load_b32(src.wsr, src.wsoff + k * 8);
    const uint32_t piece = XK == kMx4XMx4 ? lane & 7 : lane & 31;  // of 16 bytes
    const bool in_x = b + (XK == kMx4XMx4 ? piece : piece / 4) < end;
#pragma unroll
    for (int p = 0; p < PL; ++p) {
#pragma unroll
      for (int i = 0; i < NL; ++i)
        x[j][p][i] = buf_load_b128(xr, in_x ? src.xoff[i] + p * plane + b * kXBlock + piece * 16 : kOutOfRange);
    }
    if constexpr (XK == kMx4XMx4) xs[j] = buf_load_b32(xsr, xsoff + k * 8);
  }

  // The loaded step into LDS.  16-byte pieces change places within a row (4-bit:
  // piece ^ row % 8 of 8, 16-bit: piece ^ row of 32), so reads of 16 rows touch
  // all banks.
  __device__ __forceinline__ void put(int j, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) slot->w[mx4_w_row(i, lane) * 8 + ((lane & 7) ^ (lane >> 3))] = w[j][i];
    slot->ws[lane] = ws[j];
#pragma unroll
    for (int p = 0; p < PL; ++p) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int row = mx4_x_row<XK>(i, lane);
        if constexpr (XK == kMx4XMx4) slot->x[p][row * 8 + ((lane & 7) ^ (lane >> 3))] = x[j][p][i];
        else slot->x[p][row * 32 + ((lane & 31) ^ row)] = x[j][p][i];
      }
    }
    if constexpr (XK == kMx4XMx4) slot->xs[lane] = xs[j];
  }

  // The two scales of the lane's blocks of a step: those past the last column
  // (another row's) are 1, as NaN there would spoil the sum.
  __device__ __forceinline__ uint32_t scales(const uint32_t* words, int row, uint32_t skew, uint32_t k, int lane) const {
    const uint32_t g2 = 2 * (lane >> 4), b = first + k * 8 + g2;
    const uint8_t* p = reinterpret_cast<const uint8_t*>(words + 4 * row) + skew + g2;
    return (b < end ? p[0] : 127u) | (b + 1 < end ? p[1] : 127u) << 8;
  }

  // acc[0] + acc[1] += step k, which is in LDS.
  __device__ __forceinline__ void dot(float4_t* acc, uint32_t ws_skew, uint32_t k, int lane) const {
    const int r = lane & 15, g = lane >> 4, n = column;
    const uint32_t s_w = scales(slot->ws, r, ws_skew, k, lane);
    u32x4 q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) q[h] = slot->w[r * 8 + ((2 * g + h) ^ (r & 7))];
    if constexpr (XK == kMx4XMx4) {
      const uint32_t s_x = scales(slot->xs, n, xs_skew, k, lane);
      u32x4 v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) v[h] = slot->x[0][n * 8 + ((2 * g + h) ^ (n & 7))];
      acc[0] = mx4_mfma<0>(q[0], v[0], acc[0], s_w, s_x);
      acc[1] = mx4_mfma<1>(q[1], v[1], acc[1], s_w, s_x);
    } else {
      const bool fit = XK == kMx4XF16 && __ballot(!mx4_scales_fit_half(s_w)) == 0ull;
      const float s[2] = {mx4_scale<0>(s_w), mx4_scale<1>(s_w)};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t c[4] = {q[h].x, q[h].y, q[h].z, q[h].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int p = PL - 1; p >= 0; --p) {
            const u32x4 v = slot->x[p][n * 32 + ((8 * g + 4 * h + i) ^ n)];
            acc[i & 1] = mx4_mfma16<XK>(c[i], s[h], v, acc[i & 1], fit);
          }
        }
      }
    }
  }

  // Steps a wave takes of each source: whole rounds of the ring.
  __device__ __forceinline__ uint32_t turns(uint32_t stride) const {
    const uint32_t steps = (end - first + 7) / 8;
    return (steps + stride * DEPTH - 1) / (stride * DEPTH) * DEPTH;
  }
  __device__ __forceinline__ void start(const Source& src, uint32_t from, uint32_t stride, int lane) {
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) load(j, src, from + j * stride, lane);
  }
  // acc[0] + acc[1] += steps `from`, from + stride, ... of `cur`, whose first
  // ones are on their way (start, or the call before); those of `next` are when
  // it returns.
  __device__ __forceinline__ void run(float4_t* acc, const Source& cur, const Source& next, uint32_t from,
                                      uint32_t stride, int lane) {
    const uint32_t steps = (end - first + 7) / 8, n = turns(stride);
    for (uint32_t s = 0; s < n; s += DEPTH) {
#pragma unroll
      for (int j = 0; j < DEPTH; ++j) {
        const uint32_t k = from + (s + j) * stride;
        put(j, lane);
        if (s + DEPTH < n) load(j, cur, k + DEPTH * stride, lane);
        else load(j, next, from + j * stride, lane);
        wave_lds_fence();
        if (k < steps) dot(acc, cur.ws_skew, k, lane);
        wave_lds_fence();
      }
    }
  }
};

}  // namespace vqmi
