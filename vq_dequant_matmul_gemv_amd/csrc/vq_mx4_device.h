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
//   quarters of at most 36, so the 32 of a block sum exactly; the blocks and
//   the accumulator join as fp32 does: measured over every spread of the
//   scales, an instruction is off by at most 4 units of 2^-24 of the largest
//   block sum or accumulator (its products are not cut the way the e4m3
//   instructions cut theirs).
//   4-bit x 16-bit: the 4-bit values times their scale are bf16 values below
//   2^128 (infinite above), and fp16 values where the scale is between 2^-23
//   and 2^13, so one conversion per pair feeds the 16 x 16 x 32 instructions,
//   whose products are exact.  With fp16 activations, steps that hold another
//   scale take x apart into two bf16 values instead (11 bits are 8 and 3), and
//   twice the instructions.
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
// groups: 16 rows x 16 tokens x 32 columns.  x: 16-bit values, or (bf16) one of
// the planes whose sum they are.  FIT: with fp16 x, every lane's scale is one
// that fits (chosen once a step: a branch at each product took two to six times
// as long).
template <int XK, bool FIT>
__device__ __forceinline__ float4_t mx4_mfma16(uint32_t codes, float scale, u32x4 x, float4_t acc) {
  if constexpr (XK == kMx4XF16) {
    if constexpr (FIT)
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(mx4_half(codes, scale), __builtin_bit_cast(half8_t, x), acc, 0, 0,
                                                    0);
    const bf16x8_t a = mx4_bf16(codes, scale);
    bf16x8_t hi, lo;
    mx4_split_half(x, &hi, &lo);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, lo, acc, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, hi, acc, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx4_bf16(codes, scale), __builtin_bit_cast(bf16x8_t, x), acc, 0, 0,
                                                   0);
  }
}

// ---------------------------------------------------------------------------
// a wave's stream over the columns: 16 * MT rows of w, up to 16 rows of
// activations
//
// XK: what the activations are; PL: planes of them; NL: load instructions for a
// step's rows of a plane (8 rows each of 4-bit values, 2 of 16-bit ones);
// DEPTH: steps in flight.
// ---------------------------------------------------------------------------
template <int XK, int PL, int MT, int NL>
struct Mx4Slot {
  static constexpr int kRows = NL * (XK == kMx4XMx4 ? 8 : 2);  // rows of activations
  u32x4 w[MT * 16 * 8];
  u32x4 x[PL][NL * 64];
  uint32_t ws[MT * 16 * 4], xs[XK == kMx4XMx4 ? 16 * 4 : 1];  // scales: four words a row, the first two used
};

// The row a lane loads for: of w's values by instruction i, of scales by
// instruction i, and of the activations by instruction i.
__device__ __forceinline__ int mx4_w_row(int i, int lane) { return 8 * i + (lane >> 3); }
__device__ __forceinline__ int mx4_s_row(int i, int lane) { return 16 * i + (lane >> 2); }
template <int XK>
__device__ __forceinline__ int mx4_x_row(int i, int lane) {
  return XK == kMx4XMx4 ? 8 * i + (lane >> 3) : 2 * i + (lane >> 5);
}

// Scales of rows, which may start at any byte: a step's eight lie in three
// aligned words at most, which three lanes of four read.  No word without a
// byte of the tensor's is read.
struct Mx4Scales {
  const uint8_t* base;  // aligned
  uint32_t skew, bytes;
  __device__ __forceinline__ Mx4Scales(const uint8_t* p, uint32_t n)
      : base(p - (reinterpret_cast<uintptr_t>(p) & 3u)), skew((uint32_t)reinterpret_cast<uintptr_t>(p) & 3u),
        bytes((skew + n + 3u) & ~3u) {}
  // Where the scales from byte `at` of the tensor on lie: their word's offset
  // for this lane, with the bytes before them in the low two bits.
  __device__ __forceinline__ uint32_t place(uint32_t at, int lane) const {
    return (lane & 3) < 3 ? skew + at + 4 * (lane & 3) : kOutOfRange;
  }
};

// What a wave loads its steps from: rows of w and rows of activations.
template <int MT, int NL>
struct Mx4Source {
  const uint8_t *w, *ws;         // values and scales (aligned) of the rows
  uint32_t w_bytes, ws_bytes;
  uint32_t wsoff[MT], xoff[NL];  // of the lane's rows (Mx4Scales::place; bytes); kOutOfRange: no such row

  // Nothing: loads of zeros.
  __device__ __forceinline__ void clear() {
    w_bytes = ws_bytes = 0u;
#pragma unroll
    for (int i = 0; i < NL; ++i) xoff[i] = kOutOfRange;
  }
  // (member by member: as a whole the compiler copies it through memory, and
  // waits for every load in flight)
  __device__ __forceinline__ void take(const Mx4Source& o) {
    w = o.w, ws = o.ws, w_bytes = o.w_bytes, ws_bytes = o.ws_bytes;
#pragma unroll
    for (int i = 0; i < MT; ++i) wsoff[i] = o.wsoff[i];
#pragma unroll
    for (int i = 0; i < NL; ++i) xoff[i] = o.xoff[i];
  }
  // a, or b where `second` (the same in all lanes).  No branch: the loads in
  // flight stay countable.
  __device__ __forceinline__ void choose(bool second, const Mx4Source& a, const Mx4Source& b) {
    w = second ? b.w : a.w, ws = second ? b.ws : a.ws;
    w_bytes = second ? b.w_bytes : a.w_bytes, ws_bytes = second ? b.ws_bytes : a.ws_bytes;
#pragma unroll
    for (int i = 0; i < MT; ++i) wsoff[i] = second ? b.wsoff[i] : a.wsoff[i];
#pragma unroll
    for (int i = 0; i < NL; ++i) xoff[i] = second ? b.xoff[i] : a.xoff[i];
  }
};

template <int XK, int PL, int MT, int NL, int DEPTH>
struct Mx4Stream {
  typedef Mx4Slot<XK, PL, MT, NL> Slot;
  typedef Mx4Source<MT, NL> Source;
  static constexpr uint32_t kXBlock = XK == kMx4XMx4 ? 16 : 64;  // bytes of a block of activations
  rsrc_t xr, xsr;
  uint32_t woff[2 * MT], xsoff;
  uint32_t plane;       // bytes from one plane of activations to the next
  uint32_t first, end;  // blocks of columns: the first one, and behind the last
  int column;           // the row of activations that the lane multiplies
  Slot* slot;
  u32x4 w[DEPTH][2 * MT], x[DEPTH][PL][NL];
  uint32_t ws[DEPTH][MT], xs[DEPTH];

  __device__ __forceinline__ void load(int j, const Source& src, uint32_t k, int lane) {  // step k; past the end: zeros
    const uint32_t b = first + k * 8;
    const bool in_w = b + (lane & 7) < end;
    const rsrc_t wr = make_rsrc(src.w, src.w_bytes), wsr = make_rsrc(src.ws, src.ws_bytes);
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
      w[j][i] = buf_load_b128(wr, in_w ? woff[i] + b * 16 + (lane & 7) * 16 : kOutOfRange);
#pragma unroll
    for (int i = 0; i < MT; ++i) ws[j][i] = buf_load_b32(wsr, (src.wsoff[i] & ~3u) + k * 8);
    const uint32_t piece = XK == kMx4XMx4 ? lane & 7 : lane & 31;  // of 16 bytes
    const bool in_x = b + (XK == kMx4XMx4 ? piece : piece / 4) < end;
#pragma unroll
    for (int p = 0; p < PL; ++p) {
#pragma unroll
      for (int i = 0; i < NL; ++i)
        x[j][p][i] = buf_load_b128(xr, in_x ? src.xoff[i] + p * plane + b * kXBlock + piece * 16 : kOutOfRange);
    }
    if constexpr (XK == kMx4XMx4) xs[j] = buf_load_b32(xsr, (xsoff & ~3u) + k * 8);
  }

  // A row's eight scales of step k, four in each of the first two of its four
  // lanes, from the words they lie in: the next lane's word follows.  Those past
  // the last column (another row's) become 1, as NaN there would spoil the sum.
  __device__ __forceinline__ uint32_t aligned(uint32_t word, uint32_t place, uint32_t k, int lane) const {
    const uint32_t up = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)word, 0xf9, 0xf, 0xf, true);  // quad_perm 1 2 3 3
    uint32_t v = __builtin_amdgcn_alignbyte(up, word, place);
    if (first + k * 8 + 8 > end) {
      const int left = min(max((int)(end - first - k * 8) - 4 * (lane & 3), 0), 4);
      const uint32_t mask = (uint32_t)((1ull << (8 * left)) - 1ull);
      v = (v & mask) | (~mask & 0x7f7f7f7fu);
    }
    return v;
  }

  // The loaded step k into LDS.  16-byte pieces change places within a row
  // (4-bit: piece ^ row % 8 of 8, 16-bit: piece ^ row of 32), so reads of 16
  // rows touch all banks.
  __device__ __forceinline__ void put(int j, const Source& src, uint32_t k, int lane) {
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) slot->w[mx4_w_row(i, lane) * 8 + ((lane & 7) ^ (lane >> 3))] = w[j][i];
#pragma unroll
    for (int i = 0; i < MT; ++i) slot->ws[64 * i + lane] = aligned(ws[j][i], src.wsoff[i], k, lane);
#pragma unroll
    for (int p = 0; p < PL; ++p) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int row = mx4_x_row<XK>(i, lane);
        if constexpr (XK == kMx4XMx4) slot->x[p][row * 8 + ((lane & 7) ^ (lane >> 3))] = x[j][p][i];
        else slot->x[p][row * 32 + ((lane & 31) ^ row)] = x[j][p][i];
      }
    }
    if constexpr (XK == kMx4XMx4) slot->xs[lane] = aligned(xs[j], xsoff, k, lane);
  }

  // acc[m][0] + acc[m][1] += the step in LDS for rows 16 m to 16 m + 15.
  __device__ __forceinline__ void dot(float4_t (*acc)[2], int lane) const {
    const int r = lane & 15, g = lane >> 4, n = column;
    u32x4 q[MT][2];
    uint32_t s[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      s[m] = reinterpret_cast<const uint16_t*>(slot->ws + 64 * m + 4 * r)[g];
#pragma unroll
      for (int h = 0; h < 2; ++h) q[m][h] = slot->w[(16 * m + r) * 8 + ((2 * g + h) ^ (r & 7))];
    }
    if constexpr (XK == kMx4XMx4) {
      const uint32_t s_x = reinterpret_cast<const uint16_t*>(slot->xs + 4 * n)[g];
      u32x4 v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) v[h] = slot->x[0][n * 8 + ((2 * g + h) ^ (n & 7))];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        acc[m][0] = mx4_mfma<0>(q[m][0], v[0], acc[m][0], s[m], s_x);
        acc[m][1] = mx4_mfma<1>(q[m][1], v[1], acc[m][1], s[m], s_x);
      }
    } else {
      auto products = [&](auto fit) VQMI_INLINE {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u32x4 v[PL];
#pragma unroll
            for (int p = 0; p < PL; ++p) v[p] = slot->x[p][n * 32 + ((8 * g + 4 * h + i) ^ n)];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const uint32_t c = i == 0 ? q[m][h].x : i == 1 ? q[m][h].y : i == 2 ? q[m][h].z : q[m][h].w;
              const float f = h == 0 ? mx4_scale<0>(s[m]) : mx4_scale<1>(s[m]);
#pragma unroll
              for (int p = PL - 1; p >= 0; --p)
                acc[m][i & 1] = mx4_mfma16<XK, decltype(fit)::value>(c, f, v[p], acc[m][i & 1]);
            }
          }
        }
      };
      bool fit = true;
      if constexpr (XK == kMx4XF16) {
#pragma unroll
        for (int m = 0; m < MT; ++m) fit = fit && mx4_scales_fit_half(s[m]);
        fit = __ballot(!fit) == 0ull;
      }
      if (fit) products(std::true_type{});
      else if constexpr (XK == kMx4XF16) products(std::false_type{});
    }
  }

  // Steps a wave takes of each source: whole rounds of the ring.
  __device__ __forceinline__ uint32_t turns(uint32_t stride) const {
    const uint32_t steps = (end - first + 7) / 8;
    return (steps + stride * DEPTH - 1) / (stride * DEPTH) * DEPTH;
  }
  __device__ __forceinline__ void start(const Source& src, uint32_t from, uint32_t stride, int lane) {
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) {
      load(j, src, from + j * stride, lane);
      __builtin_amdgcn_sched_barrier(0);  // in the order that run() waits for them
    }
  }
  // acc += steps `from`, from + stride, ... of `cur`, whose first ones are on
  // their way (start, or the call before); those of `next` are when it returns.
  __device__ __forceinline__ void run(float4_t (*acc)[2], const Source& cur, const Source& next, uint32_t from,
                                      uint32_t stride, int lane) {
    const uint32_t steps = (end - first + 7) / 8, n = turns(stride);
    for (uint32_t s = 0; s < n; s += DEPTH) {
      const bool last = s + DEPTH >= n;
      Source src;
      src.choose(last, cur, next);
#pragma unroll
      for (int j = 0; j < DEPTH; ++j) {
        const uint32_t k = from + (s + j) * stride;
        put(j, cur, k, lane);
        __builtin_amdgcn_sched_barrier(0);
        load(j, src, last ? from + j * stride : k + DEPTH * stride, lane);
        __builtin_amdgcn_sched_barrier(0);  // the loads in their order: the next ones' wait leaves these in flight
        wave_lds_fence();
        if (k < steps) dot(acc, lane);
        wave_lds_fence();
      }
    }
  }
};

}  // namespace vqmi
