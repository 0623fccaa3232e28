// vq_store_device.h -- the output step of the block-scaled products: SwiGLU,
// rounding to y's type and the stores.  `Args` is a product's argument struct:
// y [T][rows] (rows / 2 under swiglu) of kind y_kind.
#pragma once

#include "vq_block_device.h"
#include "vq_fp8_device.h"
#include "vq_kernels.h"

#include <type_traits>

namespace vqmi {

// Eight 16-bit values as fp32.
template <bool BF16>
__device__ __forceinline__ void unpack8(u32x4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const half2_t h = __builtin_bit_cast(half2_t, w[i]);
      x[2 * i] = (float)h.x;
      x[2 * i + 1] = (float)h.y;
    }
  }
}

// silu(g) * u, silu(g) = g / (1 + exp(-g)), by the instructions for 2^x and
// 1 / x (within a unit each).  PRECISE, for an fp32 y: with e = exp(-|g|),
// g / (1 + e), or g * e / (1 + e) for a negative g, so that nothing overflows,
// and the exponent's product with log2(e) carried in two parts (one rounded
// product would cost |g| units): 6 units in all, down to g = -87.3, where silu
// is -1.1e-36 and e falls below the normal numbers: 0 from there on.  Else, for
// 16 bits, the one product, whose |g| units of 2^-24 are far below a half unit
// of 16 bits.
// (35.7 million of them behind the tile kernel at 2048 tokens, 17408 rows:
// expf() and a division 16 us, the precise form 10, the other 8.)
template <bool PRECISE>
__device__ __forceinline__ float silu_mul(float g, float u) {
  constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.69314718f;
  if constexpr (!PRECISE) return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * g)) * u;
  const float a = fminf(fabsf(g), 128.0f);  // 2^-184 is 0 already; a NaN stays in g
  const float t = a * kLog2e, low = fmaf(a, kLog2eLow, fmaf(a, kLog2e, -t));
  const float p = __builtin_amdgcn_exp2f(-t), e = fmaf(p, -kLn2 * low, p);
  return g * (g < 0.0f ? e : 1.0f) * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// N consecutive outputs, the first at y[i] (a multiple of N).
template <int N>
__device__ __forceinline__ void store_run(void* y, int64_t i, const float* v, int kind) {
  if (kind == kOutF32) {
#pragma unroll
    for (int k = 0; k < N; k += 4)
      *reinterpret_cast<float4_t*>(static_cast<float*>(y) + i + k) = float4_t{v[k], v[k + 1], v[k + 2], v[k + 3]};
    return;
  }
  uint32_t w[N / 2];
#pragma unroll
  for (int k = 0; k < N / 2; ++k) {
    w[k] = pack16(v[2 * k], v[2 * k + 1], kind == kOutF16);
  }
  uint16_t* p = static_cast<uint16_t*>(y) + i;
  if constexpr (N == 8) *reinterpret_cast<u32x4*>(p) = u32x4{w[0], w[1], w[2], w[3]};
  else *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
}

// Stores 16 tokens from t0 on of ROWS rows from r0 on (a multiple of 16) that
// lie in LDS, `pitch` floats a token; 8 rows a lane in whole pieces of y where
// its rows allow them.
template <int ROWS, bool PRECISE, typename Args>
__device__ __forceinline__ void store_tokens(const Args& a, const float* lds, int pitch, int t0, int r0, int lane) {
  if (a.rows % 8 != 0) {  // one value a lane: a token's rows still leave side by side
    auto single = [&](auto swiglu) {
      constexpr int kPairs = swiglu.value ? 2 : 1, kOut = ROWS / kPairs;
      static_assert(16 * kOut % (4 * 64) == 0, "whole rounds of the wave");
      const int rows = a.rows / kPairs, o0 = r0 / kPairs;
      for (int base = 0; base < 16 * kOut; base += 4 * 64) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = base + 64 * i + lane, k = e / kOut, o = e % kOut;
          const float* f = lds + k * pitch + kPairs * o;
          if constexpr (swiglu.value) v[i] = silu_mul<PRECISE>(f[0], f[1]);
          else v[i] = f[0];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = base + 64 * i + lane, k = e / kOut, o = e % kOut;
          if (t0 + k < a.T && o0 + o < rows) store_out(a.y, (int64_t)(t0 + k) * rows + o0 + o, v[i], a.y_kind);
        }
      }
    };
    if (a.swiglu) single(std::true_type{});
    else single(std::false_type{});
    return;
  }
  constexpr int kLanes = ROWS / 8, kPer = 64 / kLanes;  // lanes a token, tokens at once
  const int row = r0 + lane % kLanes * 8;
  if (row >= a.rows) return;
#pragma unroll 1
  for (int k = lane / kLanes; k < 16; k += kPer) {
    const int t = t0 + k;
    if (t >= a.T) break;
    const float4_t lo = *reinterpret_cast<const float4_t*>(lds + k * pitch + row - r0);
    const float4_t hi = *reinterpret_cast<const float4_t*>(lds + k * pitch + row - r0 + 4);
    if (a.swiglu) {
      const float v[4] = {silu_mul<PRECISE>(lo[0], lo[1]), silu_mul<PRECISE>(lo[2], lo[3]),
                          silu_mul<PRECISE>(hi[0], hi[1]), silu_mul<PRECISE>(hi[2], hi[3])};
      store_run<4>(a.y, (int64_t)t * (a.rows / 2) + row / 2, v, a.y_kind);
    } else {
      const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      store_run<8>(a.y, (int64_t)t * a.rows + row, v, a.y_kind);
    }
  }
}

// Four consecutive rows of one token (row: the first, a multiple of 4).
template <typename Args>
__device__ __forceinline__ void store_rows4(const Args& a, int t, int row, const float* v) {
  if (a.swiglu) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (row + 2 * p < a.rows)
        store_out(a.y, (int64_t)t * (a.rows / 2) + row / 2 + p, silu_mul<true>(v[2 * p], v[2 * p + 1]), a.y_kind);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (row + i < a.rows) store_out(a.y, (int64_t)t * a.rows + row + i, v[i], a.y_kind);
    }
  }
}

// Joining the splits of a product's columns, four values a thread of 256: y =
// the sum of the planes a.part [splits][T][rows], in their order.
template <typename Args>
__device__ __forceinline__ void join_planes(const Args& a, int splits) {
  const int64_t n = (int64_t)a.T * a.rows, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  if (n % 4 == 0 && (!a.swiglu || a.rows % 2 == 0)) {
    float4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = 0; s0 < splits; s0 += 8) {
      float4_t p[8];  // eight planes in flight
#pragma unroll
      for (int s = 0; s < 8; ++s)
        p[s] = *reinterpret_cast<const float4_t*>(a.part + min(s0 + s, splits - 1) * n + i);
#pragma unroll
      for (int s = 0; s < 8; ++s) v += s0 + s < splits ? p[s] : float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // pairs of rows never straddle a token: rows are even under SwiGLU
    if (a.swiglu) {
      store_out(a.y, i / 2, silu_mul<true>(v[0], v[1]), a.y_kind);
      store_out(a.y, i / 2 + 1, silu_mul<true>(v[2], v[3]), a.y_kind);
    } else {
      const float o[4] = {v[0], v[1], v[2], v[3]};
      store_run<4>(a.y, i, o, a.y_kind);
    }
    return;
  }
  for (int64_t k = i; k < min(n, i + 4); k += a.swiglu ? 2 : 1) {
    float v = 0.0f, u = 0.0f;
    for (int s = 0; s < splits; ++s) {
      v += a.part[s * n + k];
      if (a.swiglu) u += a.part[s * n + k + 1];
    }
    store_out(a.y, a.swiglu ? k / 2 : k, a.swiglu ? silu_mul<true>(v, u) : v, a.y_kind);
  }
}

}  // namespace vqmi
