// vq_mx4.hip -- tensors of 4-bit e2m1 values with a power-of-two scale for each
// 32 columns: quantizing, reading back, and the product.
//
//   quantize  k = floor(log2(max |x| over the block)) - 2, q = e2m1(x / 2^k)
//   product   y[t][r] = sum_b 2^(k_x[t][b] + k_w[r][b]) * sum_{c in b} q_x[t][c] * q_w[r][c],
//             or sum_c x[t][c] * w[r][c] with 16-bit x
#include "vq_block_kernels.h"
#include "vq_mx4_device.h"
#include "vq_store_device.h"

#include <type_traits>

namespace vqmi {

namespace {

// ---------------------------------------------------------------------------
// quantizer and reader: rows are whole blocks, so a tensor is one run of
// blocks of 32; 4 lanes a block, 8 values each
// ---------------------------------------------------------------------------

// Eight values at x[i], and the largest magnitude as fp32 bits.
template <int DT>
__device__ __forceinline__ uint32_t load8(const void* x, int64_t i, u32x4* raw, float* f) {
  if constexpr (DT == kOutF32) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(x) + i);
    raw[0] = p[0];
    raw[1] = p[1];
    uint32_t m = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f[k] = __uint_as_float(raw[k / 4][k % 4]);
      m = max(m, raw[k / 4][k % 4] & 0x7fffffffu);
    }
    return m;
  } else {
    raw[0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + i);
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m2 = {0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) m2 = __builtin_elementwise_max(m2, __builtin_bit_cast(u16x2, raw[0][k] & 0x7fff7fffu));
    const uint32_t m = max((uint32_t)m2.x, (uint32_t)m2.y);
    return DT == kOutBF16 ? m << 16 : __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)m));
  }
}

// The scale byte of a block whose largest magnitude has these fp32 bits:
// floor(log2) - 2 + 127, which is the exponent field less 2, at least 0; 127
// (a scale of 1) for zeros, 255 (NaN) where a value is infinite or NaN.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t top) {
  const uint32_t e = top >> 23;
  return top == 0u ? 127u : e >= 255u ? 255u : max(e, 2u) - 2u;
}

template <int DT>
__global__ __launch_bounds__(256) void vq_mx4_quant_kernel(const void* x, uint32_t* q, uint8_t* scales, int64_t pieces) {
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;  // piece of 8 values
  const bool in = p < pieces;                                 // (a multiple of 4)
  u32x4 raw[2];
  float f[8];
  uint32_t top = load8<DT>(x, (in ? p : 0) * 8, raw, f);
  // the maximum over four lanes: quad_perm 1 0 3 2 and 2 3 0 1
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xb1, 0xf, 0xf, true));
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4e, 0xf, 0xf, true));
  const uint32_t byte = mx4_scale_byte(top);
  const float s = __uint_as_float(byte << 23);
  const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
  uint32_t c = 0u;  // the conversions divide by the scale exactly, round to nearest even and stop at 6
  if constexpr (DT == kOutF32) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[0], f[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2], f[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[4], f[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[6], f[7], s, 3);
  } else if constexpr (DT == kOutF16) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(half2_t, w[0]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(half2_t, w[1]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(half2_t, w[2]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(half2_t, w[3]), s, 3);
  } else {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[0]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[1]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[2]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[3]), s, 3);
  }
  if (!in) return;
  q[p] = byte == 255u ? 0u : c;
  if ((threadIdx.x & 3u) == 0) scales[p >> 2] = (uint8_t)byte;
}

template <int DT>
__global__ __launch_bounds__(256) void vq_mx4_dequant_kernel(const uint32_t* q, const uint8_t* scales, void* y,
                                                             int64_t pieces) {
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (p >= pieces) return;
  const uint32_t c = q[p];
  const float s = __uint_as_float((uint32_t)scales[p >> 2] << 23);
  if constexpr (DT == kOutF32) {
    typedef float float2_t __attribute__((ext_vector_type(2)));
    const float2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
    const float2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
    const float2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2);
    const float2_t e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
    float4_t* o = static_cast<float4_t*>(y) + 2 * p;
    o[0] = float4_t{a.x, a.y, b.x, b.y};
    o[1] = float4_t{d.x, d.y, e.x, e.y};
  } else if constexpr (DT == kOutF16) {
    static_cast<half8_t*>(y)[p] = mx4_half(c, s);
  } else {
    static_cast<bf16x8_t*>(y)[p] = mx4_bf16(c, s);
  }
}

// ---------------------------------------------------------------------------
// product, few tokens: a block takes 16 rows of w and 16 * NT tokens, its waves
// split the columns and join their sums in LDS
// ---------------------------------------------------------------------------
struct Mx4Args {
  const uint8_t* w;
  const uint8_t* ws;
  const void* x;
  const uint8_t* xs;
  void* y;
  int rows, blocks, T;  // blocks: of 32 columns
  int y_kind, swiglu;
  int whole_w, whole_x;  // rows of scales lie on multiples of 4 bytes
  float* part;           // split columns: fp32 sums [gridDim.y][T][rows] in place of y
  int split_blocks;      // blocks of columns a split (the last one may have fewer)
};

// The arguments of one split of the columns: its sums go to their own plane of
// the workspace, as they are.
__device__ __forceinline__ Mx4Args split_args(Mx4Args a) {
  if (a.part) {
    a.y = a.part + (int64_t)blockIdx.y * a.T * a.rows;
    a.y_kind = kOutF32;
    a.swiglu = 0;
  }
  return a;
}

template <int XK, int WAVES, int NT, int PCS, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void vq_mx4_skinny_kernel(Mx4Args args) {
  const Mx4Args a = split_args(args);
  constexpr int kTok = 16 * NT, kStep = 4 * PCS;  // tokens; blocks of columns a step
  __shared__ float4_t part[WAVES][NT][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const unsigned row_tiles = (a.rows + 15) / 16;  // row tiles run fastest: they share the tokens
  const int r0 = (blockIdx.x % row_tiles) * 16, t0 = (blockIdx.x / row_tiles) * kTok;
  const int r = lane & 15, g = lane >> 4;
  const uint32_t blocks = a.blocks;
  const int rows = min(16, a.rows - r0), toks = min(kTok, a.T - t0);
  const rsrc_t wr = make_rsrc(a.w + (int64_t)r0 * blocks * 16, (uint64_t)rows * blocks * 16);
  const rsrc_t wsr = make_rsrc(a.ws + (int64_t)r0 * blocks, (uint64_t)rows * blocks);
  constexpr int kXBlock = XK == kMx4XMx4 ? 16 : 64;  // bytes of a block of activations
  const rsrc_t xr = make_rsrc(static_cast<const uint8_t*>(a.x) + (int64_t)t0 * blocks * kXBlock,
                              (uint64_t)toks * blocks * kXBlock);
  const rsrc_t xsr = make_rsrc(XK == kMx4XMx4 ? a.xs + (int64_t)t0 * blocks : nullptr, (uint64_t)toks * blocks);
  const uint32_t wrow = r < rows ? (uint32_t)r : kOutOfRange;
  uint32_t xrow[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint32_t t = 16 * n + r;
    xrow[n] = t < (uint32_t)toks ? (XK == kMx4XMx4 ? t : t * blocks * kXBlock) : kOutOfRange;
  }
  float4_t acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  Mx4Step<XK, PCS, NT> st[DEPTH];
  const uint32_t b_first = blockIdx.y * a.split_blocks, b_end = min(blocks, b_first + a.split_blocks);
  auto load = [&](int j, uint32_t k) {  // steps past the end: zeros
    const uint32_t b = b_first + k * kStep + g * PCS;
    mx4_load(st[j].w, wr, wsr, wrow, b, b_end, blocks, a.whole_w);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (XK == kMx4XMx4) mx4_load(st[j].x[n], xr, xsr, xrow[n], b, b_end, blocks, a.whole_x);
      else mx4_load_x(st[j].x[n], xr, xrow[n], 0u, b, b_end);
    }
  };
  const uint32_t steps = (b_end - b_first + kStep - 1) / kStep;
#pragma unroll
  for (int j = 0; j < DEPTH; ++j) load(j, wave + j * WAVES);
  for (uint32_t k = wave; k < steps; k += DEPTH * WAVES) {
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) {  // no branches: the loads in flight are counted through the loop
      st[j].dot(acc);
      load(j, k + (j + DEPTH) * WAVES);
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) part[wave][n][lane] = acc[n];
  __syncthreads();
  if (wave >= NT) return;  // wave n joins token tile n
  float4_t sum = part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) sum += part[w][wave][lane];
  const int t = t0 + 16 * wave + r;
  const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
  if (t < a.T) store_rows4(a, t, r0 + g * 4, v);
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <int XK, int WAVES, int NT, int PCS, int DEPTH>
void run_skinny(const Mx4Args& a, int splits, hipStream_t s) {
  const dim3 grid((unsigned)ceil_div(a.rows, 16) * ceil_div(a.T, 16 * NT), splits);
  hipLaunchKernelGGL((vq_mx4_skinny_kernel<XK, WAVES, NT, PCS, DEPTH>), grid, dim3(64 * WAVES), 0, s, a);
}

template <int XK>
void run_kind(const Mx4Args& a, hipStream_t s) {
  if (a.T <= 16) return run_skinny<XK, 4, 1, 2, 2>(a, 1, s);
  if (a.T <= 32) return run_skinny<XK, 4, 2, 1, 2>(a, 1, s);
  run_skinny<XK, 4, 4, 1, 2>(a, 1, s);
}

}  // namespace

hipError_t launch_mx4_quant(const void* x, int x_kind, int64_t values, uint8_t* q, uint8_t* scales, hipStream_t s) {
  const int64_t pieces = values / 8;
  const dim3 grid((unsigned)((pieces + 255) / 256)), block(256);
  uint32_t* qw = reinterpret_cast<uint32_t*>(q);
  if (x_kind == kOutF32) hipLaunchKernelGGL((vq_mx4_quant_kernel<kOutF32>), grid, block, 0, s, x, qw, scales, pieces);
  else if (x_kind == kOutF16) hipLaunchKernelGGL((vq_mx4_quant_kernel<kOutF16>), grid, block, 0, s, x, qw, scales, pieces);
  else hipLaunchKernelGGL((vq_mx4_quant_kernel<kOutBF16>), grid, block, 0, s, x, qw, scales, pieces);
  return hipGetLastError();
}

hipError_t launch_mx4_dequant(const uint8_t* q, const uint8_t* scales, int64_t values, void* y, int y_kind,
                              hipStream_t s) {
  const int64_t pieces = values / 8;
  const dim3 grid((unsigned)((pieces + 255) / 256)), block(256);
  const uint32_t* qw = reinterpret_cast<const uint32_t*>(q);
  if (y_kind == kOutF32) hipLaunchKernelGGL((vq_mx4_dequant_kernel<kOutF32>), grid, block, 0, s, qw, scales, y, pieces);
  else if (y_kind == kOutF16) hipLaunchKernelGGL((vq_mx4_dequant_kernel<kOutF16>), grid, block, 0, s, qw, scales, y, pieces);
  else hipLaunchKernelGGL((vq_mx4_dequant_kernel<kOutBF16>), grid, block, 0, s, qw, scales, y, pieces);
  return hipGetLastError();
}

Mx4Plans mx4_plans(int rows, int cols, int T) {
  Mx4Plan p;
  const int64_t tiles = (int64_t)ceil_div(rows, 16) * ceil_div(T, T <= 16 ? 16 : T <= 32 ? 32 : 64);
  p.kernel = tiles < (1 << 24) ? 0 : -1;
  return {p, p};
}

hipError_t launch_mx4_gemm(const Mx4View& w, const IoSpec& io, const Mx4Plan& p, const void* x, int x_kind,
                           const uint8_t* xs, int T, void* y, void* workspace, hipStream_t s) {
  Mx4Args a{};
  a.w = w.values;
  a.ws = w.scales;
  a.x = x;
  a.xs = xs;
  a.y = y;
  a.rows = w.rows;
  a.blocks = w.cols / kMx4Block;
  a.T = T;
  a.y_kind = io.y_kind;
  a.swiglu = io.epi == kEpiSwiglu;
  auto whole = [&](const uint8_t* q) { return a.blocks % 4 == 0 && reinterpret_cast<uintptr_t>(q) % 4 == 0; };
  a.whole_w = whole(w.scales);
  a.whole_x = whole(xs);
  a.split_blocks = a.blocks;
  if (x_kind == kMx4XMx4) run_kind<kMx4XMx4>(a, s);
  else if (x_kind == kMx4XF16) run_kind<kMx4XF16>(a, s);
  else run_kind<kMx4XBF16>(a, s);
  return hipGetLastError();
}

}  // namespace vqmi
