// vq_mx4.hip -- tensors of 4-bit e2m1 values with a power-of-two scale for each
// 32 columns: quantizing, reading back, and the product.
//
//   quantize  k = floor(log2(max |x| over the block)) - 2, q = e2m1(x / 2^k)
//   product   y[t][r] = sum_b 2^(k_x[t][b] + k_w[r][b]) * sum_{c in b} q_x[t][c] * q_w[r][c],
//             or sum_c x[t][c] * w[r][c] with 16-bit x
#include "vq_block_kernels.h"
#include "vq_mx4_device.h"
#include "vq_store_device.h"

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <type_traits>

namespace vqmi {

namespace {

// ---------------------------------------------------------------------------
// quantizer and reader: rows are whole blocks, so a tensor is one run of
// blocks of 32; 4 lanes a block, 8 values (16 bytes of 16-bit x) each, the
// block's maximum by two lane exchanges.  Bound by memory: 4096 x 5120 fp16
// values take 10.0 us each way, 5.3 TB/s, a large copy's rate; 4 x 17408 bf16
// values 2.8, which is a launch.
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
__global__ __launch_bounds__(256) void vq_mx4_quant_kernel(const void* x, uint32_t* q, uint8_t* scales,
                                                           int64_t pieces) {
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
// product, few tokens: a block takes 16 rows of w (or 32) and up to 16 tokens,
// its waves split the columns and join their sums in LDS
//
// Bound by the weight's bytes: one token of 17408 x 5120 (47 MB) takes 12.7 us
// with 4-bit x and 13.0 with bf16 x, 3.7 TB/s; less the launch's 2.3 us that is
// 4.5 TB/s of a copy's 5.2.  Waves that stream rows' columns through LDS of
// their own need no barrier until the end; fragments loaded straight from memory
// took 18 us, and more than two steps in flight gained nothing.
// ---------------------------------------------------------------------------
struct Mx4Args {
  const uint8_t* w;
  const uint8_t* ws;
  const void* x;
  const uint8_t* xs;
  void* y;
  int rows, blocks, T;  // blocks: of 32 columns
  int y_kind, swiglu;
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

template <int XK, int WAVES, int MT, int NL, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void vq_mx4_skinny_kernel(Mx4Args args) {
  const Mx4Args a = split_args(args);
  typedef Mx4Stream<XK, 1, MT, NL, DEPTH> Stream;
  constexpr int kTok = Stream::Slot::kRows, kRows = 16 * MT;
  __shared__ typename Stream::Slot slots[WAVES];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const unsigned row_tiles = (a.rows + kRows - 1) / kRows;  // row tiles run fastest: they share the tokens
  const int r0 = (blockIdx.x % row_tiles) * kRows, t0 = (blockIdx.x / row_tiles) * kTok;
  const int r = lane & 15, g = lane >> 4;
  const uint32_t blocks = a.blocks;
  const int rows = min(kRows, a.rows - r0), toks = min(kTok, a.T - t0);
  Stream st;
  st.slot = slots + wave;
  st.first = blockIdx.y * a.split_blocks;
  st.end = min(blocks, st.first + a.split_blocks);
  typename Stream::Source src;
  src.w = a.w + (int64_t)r0 * blocks * 16;
  src.w_bytes = rows * blocks * 16;
  st.xr = make_rsrc(static_cast<const uint8_t*>(a.x) + (int64_t)t0 * blocks * Stream::kXBlock,
                    (uint64_t)toks * blocks * Stream::kXBlock);
  st.plane = 0;
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
    const int row = mx4_w_row(i, lane);
    st.woff[i] = row < rows ? row * blocks * 16 : kOutOfRange;
  }
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int row = mx4_x_row<XK>(i, lane);
    src.xoff[i] = row < toks ? row * blocks * Stream::kXBlock : kOutOfRange;
  }
  st.column = r & (kTok - 1);
  const Mx4Scales ws(a.ws + (int64_t)r0 * blocks, rows * blocks);
  src.ws = ws.base;
  src.ws_bytes = ws.bytes;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    // rows past the end take the last one's: zeros would not fit fp16
    src.wsoff[i] = ws.place(min(mx4_s_row(i, lane), rows - 1) * blocks + st.first, lane);
  }
  if constexpr (XK == kMx4XMx4) {
    const Mx4Scales xs(a.xs + (int64_t)t0 * blocks, toks * blocks);
    st.xsr = make_rsrc(xs.base, xs.bytes);
    st.xsoff = mx4_s_row(0, lane) < toks ? xs.place(mx4_s_row(0, lane) * blocks + st.first, lane) : kOutOfRange;
  }
  float4_t acc[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  st.start(src, wave, WAVES, lane);
  typename Stream::Source none;
  none.take(src);
  none.clear();
  st.run(acc, src, none, wave, WAVES, lane);
  __syncthreads();  // the slots are free: the waves' sums go there
  float4_t* part = reinterpret_cast<float4_t*>(slots);
  static_assert(sizeof(slots) >= WAVES * MT * 64 * sizeof(float4_t), "every wave's sums fit");
#pragma unroll
  for (int m = 0; m < MT; ++m) part[(wave * MT + m) * 64 + lane] = acc[m][0] + acc[m][1];
  __syncthreads();
  if (wave >= MT) return;  // wave m joins row tile m
  float4_t sum = part[wave * 64 + lane];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) sum += part[(w * MT + wave) * 64 + lane];
  const int t = t0 + r;
  const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
  if (r < toks) store_rows4(a, t, r0 + wave * 16 + g * 4, v);
}

// The sums of KW groups of kWaves waves, joined in their order by the first
// group through each other's LDS (free now; at(group): where it is).  False for
// the others, which are done.
template <int KW, int WAVES, int MT, int NT, typename At>
__device__ __forceinline__ bool join_groups(float4_t (&acc)[MT][NT], int group, int wave, int lane, At at) {
  const int first = wave * MT * NT * 64 + lane;
  if (group > 0) {
    float4_t* part = reinterpret_cast<float4_t*>(at(group));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int n = 0; n < NT; ++n) part[first + (m * NT + n) * 64] = acc[m][n];
    }
  }
  __syncthreads();
  if (group > 0) return false;
#pragma unroll
  for (int o = 1; o < KW; ++o) {
    const float4_t* part = reinterpret_cast<const float4_t*>(at(o));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] += part[first + (m * NT + n) * 64];
    }
  }
  return true;
}

// ---------------------------------------------------------------------------
// product, many tokens, 4-bit x: WM x WN waves of 16*MT rows x 16*NT tokens a
// block, steps of 256 columns (8 blocks, 128 bytes a row); with KW > 1 that many
// groups of such waves split a block's columns, for products of too few tiles to
// fill the card otherwise (128 tokens of 5120 x 5120: 17.3 us with splits that a
// second launch joins, 13.5 with two groups)
//
// 2048 tokens of 17408 x 5120 with SwiGLU take 114 to 123 us, 3.0 to 3.2 PF/s;
// 4096 of 8192 x 8192 139 to 150 us, 3.7 to 3.9 PF/s.  Bound by the matrix instructions at the card's power
// limit, then by the loads and their way through LDS: of 139 us that the latter
// takes in a warm loop they alone run 96; without the loads and their writes to LDS
// it takes 115, without the loads 122, without scales 129, without fragment reads
// 130 (parts left out of a copy of this kernel; the 2048 tokens without SwiGLU
// 129, 93 alone, 110, 119, 120 and 121).  Loads straight into LDS, three steps
// ahead, were slower: a block on its own took 141 us where this takes 104.
// ---------------------------------------------------------------------------
template <bool PRECISE, int WM, int WN, int MT, int NT, int KW>
__global__ __launch_bounds__(64 * WM * WN * KW, WM * WN * KW / 4) void vq_mx4_tile_kernel(Mx4Args args) {
  const Mx4Args a = split_args(args);
  constexpr int kWaves = WM * WN, kTileRows = 16 * MT * WM, kTileTokens = 16 * NT * WN;
  constexpr int kLoadRows = 8 * kWaves;  // rows the block loads at once
  constexpr int kWLoads = kTileRows / kLoadRows, kXLoads = kTileTokens / kLoadRows, kLoads = kWLoads + kXLoads;
  static_assert(kTileRows % kLoadRows == 0 && kTileTokens % kLoadRows == 0, "whole loads");
  static_assert(kTileRows + kTileTokens <= 64 * kWaves && kTileRows % 64 == 0 && kTileTokens % 32 == 0,
                "a thread loads one row's scales, a wave those of one operand");
  static_assert(NT % 2 == 0, "two token operands in turn");
  __shared__ __align__(1024) uint8_t lds_w_all[KW][2][kTileRows * 128];
  __shared__ __align__(1024) uint8_t lds_x_all[KW][2][kTileTokens * 128];
  __shared__ __align__(1024) u32x4 lds_s_all[KW][2][64 * kWaves];  // scales of two steps, a row a thread, twice
  const int group = KW == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / kWaves;  // of the columns
  const uint32_t thread = threadIdx.x - group * 64 * kWaves;
  const int wave = __builtin_amdgcn_readfirstlane(thread >> 6), lane = thread & 63;
  uint8_t(*lds_w)[kTileRows * 128] = lds_w_all[group];
  uint8_t(*lds_x)[kTileTokens * 128] = lds_x_all[group];
  u32x4(*lds_s)[64 * kWaves] = lds_s_all[group];
  const uint32_t blocks = a.blocks, pitch = blocks * 16;
  const int row_tiles = (a.rows + kTileRows - 1) / kTileRows, tok_tiles = (a.T + kTileTokens - 1) / kTileTokens;
  int rt, tt;
  xcd_tile(blockIdx.x, row_tiles, tok_tiles, &rt, &tt);
  const int r0 = rt * kTileRows, t0 = tt * kTileTokens;
  const int rows = min(kTileRows, a.rows - r0), toks = min(kTileTokens, a.T - t0);
  const rsrc_t wr = make_rsrc(a.w + (int64_t)r0 * pitch, (uint64_t)rows * pitch);
  const rsrc_t xr = make_rsrc(static_cast<const uint8_t*>(a.x) + (int64_t)t0 * pitch, (uint64_t)toks * pitch);
  const int wm = wave / WN * 16 * MT, wn = wave % WN * 16 * NT;  // the wave's rows and tokens

  // A wave loads 8 rows of 128 bytes at a time, 16 bytes a lane, through
  // registers into LDS.  The 16-byte pieces (blocks of 32 columns) of row r lie
  // in the order piece ^ (r % 8), so the fragment reads of 8 rows touch all
  // banks.  Columns, rows and steps past the end arrive as zeros.
  const uint32_t ld_piece = lane & 7, ld_row = wave * 8 + (lane >> 3);
  const uint32_t ld_dst = ld_row * 128 + ((ld_piece ^ (lane >> 3)) * 16);
  const uint32_t s0 = blockIdx.y * a.split_blocks, s1 = min(blocks, s0 + a.split_blocks);  // s0: a multiple of 16
  const uint32_t pairs = ((s1 - s0 + 15) / 16 + KW - 1) / KW;  // steps of each group, taken two by two
  const uint32_t b0 = s0 + group * pairs * 16, b1 = min(s1, b0 + pairs * 16);  // b1 <= b0: nothing left
  u32x4 stage[kLoads];
  auto stage_off = [&](uint32_t s) {
    const uint32_t b = b0 + s * 8 + ld_piece;
    return b < b1 ? ld_row * pitch + b * 16 : kOutOfRange;
  };
  auto load_piece = [&](uint32_t off, int i) {
    stage[i] = i < kWLoads ? buf_load_b128(wr, off + i * kLoadRows * pitch)
                           : buf_load_b128(xr, off + (i - kWLoads) * kLoadRows * pitch);
  };
  auto write_piece = [&](uint32_t s, int i) {
    uint8_t* to = i < kWLoads ? lds_w[s & 1] + i * kLoadRows * 128 : lds_x[s & 1] + (i - kWLoads) * kLoadRows * 128;
    *reinterpret_cast<u32x4*>(to + ld_dst) = stage[i];
  };
  // The 16 scales of a row's two steps, a row a thread, as the aligned words
  // they lie in (rows of scales start at any byte; no word without a byte of
  // the tensor's is read).  Lane group g of a fragment takes blocks 2g and 2g +
  // 1 of a step, so dword g holds those of the first step, then those of the
  // second.  Scales past the last column are zeros: another row's there might
  // be NaN.
  const bool sc_w = wave * 64 < kTileRows;  // waves load either operand's
  const uint8_t* sc_base = sc_w ? a.ws + (int64_t)r0 * blocks : a.xs + (int64_t)t0 * blocks;
  const uint32_t sc_skew = (uint32_t)reinterpret_cast<uintptr_t>(sc_base) & 3u, sc_rows = sc_w ? rows : toks;
  const uint32_t sc_words = (sc_skew + sc_rows * blocks + 3) / 4;
  const rsrc_t sr = make_rsrc(sc_base - sc_skew, (uint64_t)sc_words * 4);
  const uint32_t sc_row = sc_w ? thread : thread - kTileRows;
  const uint32_t sc_off = sc_skew + sc_row * blocks + b0;
  const bool sc_live = sc_row < sc_rows;
  int sc_left = (int)(b1 - b0);  // scales from the next ones to be written on
  // (in vector registers: scalar compares keep the compiler from interleaving what follows)
  asm("" : "+v"(sc_left));
  uint32_t stage_s[5];
  auto load_scales = [&](uint32_t v) VQMI_INLINE {
    const uint32_t off = sc_live ? (sc_off + v * 16) & ~3u : kOutOfRange;
#pragma unroll
    for (int i = 0; i < 5; ++i) stage_s[i] = buf_load_b32(sr, off + 4 * i);
  };
  auto write_scales = [&](uint32_t v) VQMI_INLINE {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int left = min(max(sc_left - 4 * i, 0), 4);  // of this word
      w[i] = __builtin_amdgcn_alignbyte(stage_s[i + 1], stage_s[i], sc_off) & (uint32_t)((1ull << (8 * left)) - 1ull);
    }
    sc_left -= 16;
    // (no branch: the compiler would move matrix instructions past it)
    lds_s[v & 1][thread] = u32x4{(w[0] & 0xffffu) | w[2] << 16, w[0] >> 16 | (w[2] & 0xffff0000u),
                                      (w[1] & 0xffffu) | w[3] << 16, w[1] >> 16 | (w[3] & 0xffff0000u)};
  };
  const int r = lane & 15, g = lane >> 4;
  const uint32_t f_lo = r * 128 + (((2 * g) ^ (r & 7)) * 16), f_hi = r * 128 + (((2 * g + 1) ^ (r & 7)) * 16);
  struct Op {
    u32x4 lo, hi;
  };
  auto read_lo = [&](Op& o, const uint8_t* base) { o.lo = *reinterpret_cast<const u32x4*>(base + f_lo); };
  auto read_hi = [&](Op& o, const uint8_t* base) { o.hi = *reinterpret_cast<const u32x4*>(base + f_hi); };
  auto read_scale = [&](uint32_t v, int row) {  // row: of the rows, then of the tokens
    return reinterpret_cast<const uint32_t*>(&lds_s[v & 1][row + r])[g];
  };

  float4_t acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // The first step in LDS, the second in registers; the first two steps' scales
  // in LDS, the next two's in registers.
  load_scales(0);
#pragma unroll
  for (uint32_t s = 0; s < 2; ++s) {
    const uint32_t off = stage_off(s);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load_piece(off, i);
    if (s < 1) {
      write_scales(0);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) write_piece(s, i);
    }
  }
  load_scales(1);
  lds_barrier();
  Op av[MT], bv[2];  // token operands: the current one and the next
  uint32_t sa[MT], sb[NT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    read_lo(av[m], lds_w[0] + (wm + 16 * m) * 128);
    read_hi(av[m], lds_w[0] + (wm + 16 * m) * 128);
    sa[m] = read_scale(0, wm + 16 * m);
  }
  read_lo(bv[0], lds_x[0] + wn * 128);
  read_hi(bv[0], lds_x[0] + wn * 128);
#pragma unroll
  for (int n = 0; n < NT; ++n) sb[n] = read_scale(0, kTileRows + wn + 16 * n);

  auto step = [&](uint32_t v, auto parity) VQMI_INLINE {
    constexpr int P = parity.value;
    const uint32_t s = 2 * v + P;
    const uint8_t* xb = lds_x[P] + wn * 128;
    const uint8_t* xnext = lds_x[P ^ 1] + wn * 128;
    const uint8_t* wnext = lds_w[P ^ 1] + wm * 128;
    const uint32_t off = stage_off(s + 2);
    uint32_t sb_next[NT];
    static_for<NT>([&](auto nc) VQMI_INLINE {
      constexpr int n = nc.value;
      // every wave has issued its last reads of this step before the barrier
      // waits for them, so behind it the next step's pieces in LDS are complete
      // and this one's buffers free
      if constexpr (n == NT - 1) lds_barrier();
      const uint8_t* from = (n + 1 < NT ? xb : xnext) + (n + 1) % NT * 16 * 128;
      read_lo(bv[(n + 1) % 2], from);
      read_hi(bv[(n + 1) % 2], from);
      static_for<2 * MT>([&](auto hm) VQMI_INLINE {
        constexpr int h = hm.value / MT, m = hm.value % MT;
        const Op& b = bv[n % 2];
        if constexpr (h == 0) acc[m][n] = mx4_mfma<2 * P>(av[m].lo, b.lo, acc[m][n], sa[m], sb[n]);
        else acc[m][n] = mx4_mfma<2 * P + 1>(av[m].hi, b.hi, acc[m][n], sa[m], sb[n]);
        __builtin_amdgcn_sched_barrier(0);
        // the next step's pieces go to LDS, spread over the step, and the ones
        // after them are loaded in their place
        constexpr int kSlots = (NT - 1) * MT * 2, i = n * 2 * MT + hm.value;
        static_for<kLoads>([&](auto k) VQMI_INLINE {
          if constexpr (k.value * kSlots / kLoads == i) {
            write_piece(s + 1, k.value);
            load_piece(off, k.value);
          }
        });
        // the next two steps' scales: written before the odd step's barrier
        if constexpr (P == 0 && i == 0) write_scales(v + 1);
        if constexpr (P == 0 && i == kSlots) load_scales(v + 2);
        if constexpr (n == NT - 1) {
          if constexpr (h == 0) read_lo(av[m], wnext + m * 16 * 128);
          else read_hi(av[m], wnext + m * 16 * 128);
          if constexpr (P == 1 && h == 1) {
            sa[m] = read_scale(v + 1, wm + 16 * m);
#pragma unroll
            for (int k = m; k < NT; k += MT) sb_next[k] = read_scale(v + 1, kTileRows + wn + 16 * k);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    if constexpr (P == 1) {
#pragma unroll
      for (int n = 0; n < NT; ++n) sb[n] = sb_next[n];
    }
  };
  const uint32_t steps = KW == 1 ? (b1 - b0 + 7) / 8 : 2 * pairs;  // (the barriers are every group's)
  for (uint32_t v = 0; v < pairs; ++v) {
    step(v, std::integral_constant<int, 0>{});
    if (2 * v + 1 < steps) step(v, std::integral_constant<int, 1>{});
  }
  // The waves' outputs go through the same LDS, 16 tokens at a time, so that a
  // token's rows leave in whole pieces.
  lds_barrier();
  if constexpr (KW > 1) {
    if (!join_groups<KW, kWaves, MT, NT>(acc, group, wave, lane, [&](int o) VQMI_INLINE { return lds_w_all[o][0]; }))
      return;
  }
  constexpr int kPitch = 16 * MT + 4;  // fp32 a token
  static_assert(kWaves * 16 * kPitch * 4 <= (int)sizeof(lds_w_all[0]), "every wave's 16 tokens fit");
  static_assert(KW == 1 || kWaves * MT * NT * 1024 <= (int)sizeof(lds_w_all[0]), "a group's sums fit");
  float* out = reinterpret_cast<float*>(&lds_w[0][0]) + wave * 16 * kPitch;
  static_for<NT>([&](auto n) VQMI_INLINE {
#pragma unroll
    for (int m = 0; m < MT; ++m) *reinterpret_cast<float4_t*>(out + r * kPitch + 16 * m + 4 * g) = acc[m][n.value];
    wave_lds_fence();
    store_tokens<16 * MT, PRECISE>(a, out, kPitch, t0 + wn + 16 * n.value, r0 + wm, lane);
    wave_lds_fence();
  });
}

// ---------------------------------------------------------------------------
// product, many tokens, 16-bit x: WM x WN waves of 16*MT rows x 16*NT tokens a
// block, steps of 128 columns (4 blocks: 64 bytes a row of w, 256 a token), KW
// groups of them as above
//
// 61 tokens of 5121 x 4096 take 15.1 us, bound by the latency of a step, of which
// four groups of waves overlap some (17.4 us in one, with splits): the loads' way
// through LDS first, without which a copy took 10.4 (12.3 without the loads alone),
// then conversions (14.3 without) and the reads of x (14.0), 9.5 without all four.
// (4-bit x in the kernel above, two groups of 64 x 64: 15.1, without the same 11.5,
// the loads 12.5, scales 13.4, fragment reads 15.1, all 10.7.)
// 2048 tokens of 17408 x 5120 take 360 to 378 us, 1.0 PF/s, bound by the LDS traffic of
// 16-bit x beside the matrix instructions.
// ---------------------------------------------------------------------------
template <int XK, bool PRECISE, int WM, int WN, int MT, int NT, int KW>
__global__ __launch_bounds__(64 * WM * WN * KW) void vq_mx4_tile16_kernel(Mx4Args args) {
  const Mx4Args a = split_args(args);
  constexpr int kWaves = WM * WN, kTileRows = 16 * MT * WM, kTileTokens = 16 * NT * WN;
  constexpr int kWLoads = kTileRows / (16 * kWaves), kXLoads = kTileTokens / (4 * kWaves);  // a wave: 16 rows, 4 tokens
  static_assert(kTileRows % (16 * kWaves) == 0 && kTileTokens % (4 * kWaves) == 0, "whole loads");
  constexpr int kTileBytes = kTileRows * 64 + kTileTokens * 256;
  constexpr int kPitch = 16 * MT + 4;  // of the outputs in LDS: fp32 a token
  constexpr int kOutBytes = kWaves * 16 * kPitch * 4;
  static_assert(2 * kTileBytes >= kOutBytes && (KW == 1 || 2 * kTileBytes >= kWaves * MT * NT * 1024), "outputs fit");
  __shared__ __align__(1024) uint8_t lds_all[KW][2 * kTileBytes];
  __shared__ uint32_t lds_s_all[KW][2][kTileRows];  // a row's scales of a step
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / kWaves;  // of the columns
  const int thread = threadIdx.x - group * 64 * kWaves, lane = thread & 63;
  const int wave = __builtin_amdgcn_readfirstlane(thread >> 6);
  uint8_t* lds = lds_all[group];
  uint32_t(*lds_s)[kTileRows] = lds_s_all[group];
  const uint32_t blocks = a.blocks;
  const int row_tiles = (a.rows + kTileRows - 1) / kTileRows, tok_tiles = (a.T + kTileTokens - 1) / kTileTokens;
  int rt, tt;
  xcd_tile(blockIdx.x, row_tiles, tok_tiles, &rt, &tt);
  const int r0 = rt * kTileRows, t0 = tt * kTileTokens;
  const int rows = min(kTileRows, a.rows - r0), toks = min(kTileTokens, a.T - t0);
  const rsrc_t wr = make_rsrc(a.w + (int64_t)r0 * blocks * 16, (uint64_t)rows * blocks * 16);
  const rsrc_t xr =
      make_rsrc(static_cast<const uint8_t*>(a.x) + (int64_t)t0 * blocks * 64, (uint64_t)toks * blocks * 64);
  const int wm = wave / WN * 16 * MT, wn = wave % WN * 16 * NT;
  const uint32_t s0 = blockIdx.y * a.split_blocks, s1 = min(blocks, s0 + a.split_blocks);
  const uint32_t steps = ((s1 - s0 + 3) / 4 + KW - 1) / KW;  // of each group
  const uint32_t b0 = s0 + group * steps * 4, b1 = min(s1, b0 + steps * 4);  // b1 < b0: nothing left

  // 16-byte pieces change places within a row (w: piece ^ row / 2 of 4, x: piece
  // ^ token of 16), so reads of 16 rows touch all banks.
  const uint32_t w_row = wave * 16 + (lane >> 2), w_piece = lane & 3;
  const uint32_t x_row = wave * 4 + (lane >> 4), x_piece = lane & 15;
  u32x4 sw[kWLoads], sx[kXLoads];  // the step on its way
  uint32_t ss[2];
  // scales of row threadIdx.x, as the two aligned words that a step's four lie in
  const uint8_t* sc_base = a.ws + (int64_t)r0 * blocks;
  const uint32_t sc_skew = (uint32_t)reinterpret_cast<uintptr_t>(sc_base) & 3u;
  const rsrc_t sr = make_rsrc(sc_base - sc_skew, (uint64_t)((sc_skew + (uint64_t)rows * blocks + 3) & ~3ull));
  static_assert(kTileRows <= 64 * kWaves, "a thread loads one row's scales");
  // (rows past the end take the last one's: zeros would not fit fp16)
  const uint32_t sc_off = sc_skew + min(thread, rows - 1) * blocks + b0;
  auto load = [&](uint32_t s) VQMI_INLINE {  // past the end: zeros
    const uint32_t bw = b0 + s * 4 + w_piece, bx = b0 + s * 4 + x_piece / 4;
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
      sw[i] = buf_load_b128(wr, bw < b1 ? ((w_row + i * 16 * kWaves) * blocks + bw) * 16 : kOutOfRange);
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
      sx[i] = buf_load_b128(
          xr, bx < b1 ? ((x_row + i * 4 * kWaves) * blocks + b0 + s * 4) * 64 + x_piece * 16 : kOutOfRange);
    const uint32_t off = (sc_off + s * 4) & ~3u;
    ss[0] = buf_load_b32(sr, off);
    ss[1] = buf_load_b32(sr, off + 4);
    __builtin_amdgcn_sched_barrier(0);  // in the order that they are waited for
  };
  auto put = [&](uint32_t s) VQMI_INLINE {
    uint8_t* to = lds + (s & 1) * kTileBytes;
#pragma unroll
    for (int i = 0; i < kWLoads; ++i) {
      const uint32_t row = w_row + i * 16 * kWaves;
      *reinterpret_cast<u32x4*>(to + row * 64 + ((w_piece ^ (row >> 1 & 3)) * 16)) = sw[i];
    }
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
      const uint32_t row = x_row + i * 4 * kWaves;
      *reinterpret_cast<u32x4*>(to + kTileRows * 64 + row * 256 + ((x_piece ^ (row & 15)) * 16)) = sx[i];
    }
    if (thread < kTileRows) {
      // scales past the last column (another row's) are 1: NaN there would spoil the sum
      const int left = (int)(b1 - b0) - (int)(4 * s);
      const uint32_t mask = left >= 4 ? ~0u : (1u << (8 * max(left, 0))) - 1u;
      lds_s[s & 1][thread] = (__builtin_amdgcn_alignbyte(ss[1], ss[0], sc_off) & mask) | (~mask & 0x7f7f7f7fu);
    }
  };
  const int r = lane & 15, g = lane >> 4;
  float4_t acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  load(0);
  put(0);
  load(1);
  lds_barrier();
  for (uint32_t s = 0; s < steps; ++s) {
    const uint8_t* wb = lds + (s & 1) * kTileBytes + (wm + r) * 64 + ((g ^ (r >> 1 & 3)) * 16);
    const uint8_t* xb = lds + (s & 1) * kTileBytes + kTileRows * 64 + (wn + r) * 256;
    u32x4 q[MT];
    float sc[MT];
    bool fit = true;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      q[m] = *reinterpret_cast<const u32x4*>(wb + m * 16 * 64);
      const uint32_t byte = reinterpret_cast<const uint8_t*>(&lds_s[s & 1][wm + 16 * m + r])[g];
      sc[m] = __uint_as_float(byte << 23);
      fit = fit && byte - 104u <= 36u;
    }
    fit = XK == kMx4XBF16 || __ballot(!fit) == 0ull;
    put(s + 1);
    load(s + 2);
    auto products = [&](auto fit) VQMI_INLINE {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u32x4 v[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
          v[n] = *reinterpret_cast<const u32x4*>(xb + n * 16 * 256 + (((4 * g + i) ^ r) * 16));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint32_t c = i == 0 ? q[m].x : i == 1 ? q[m].y : i == 2 ? q[m].z : q[m].w;
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[m][n] = mx4_mfma16<XK, decltype(fit)::value>(c, sc[m], v[n], acc[m][n]);
        }
      }
    };
    if (fit) products(std::true_type{});
    else if constexpr (XK == kMx4XF16) products(std::false_type{});
    lds_barrier();
  }
  if constexpr (KW > 1) {
    if (!join_groups<KW, kWaves, MT, NT>(acc, group, wave, lane, [&](int o) VQMI_INLINE { return lds_all[o]; })) return;
  }
  // The waves' outputs go through the same LDS, 16 tokens at a time, so that a
  // token's rows leave in whole pieces.
  float* out = reinterpret_cast<float*>(lds) + wave * 16 * kPitch;
  static_for<NT>([&](auto n) VQMI_INLINE {
#pragma unroll
    for (int m = 0; m < MT; ++m) *reinterpret_cast<float4_t*>(out + r * kPitch + 16 * m + 4 * g) = acc[m][n.value];
    wave_lds_fence();
    store_tokens<16 * MT, PRECISE>(a, out, kPitch, t0 + wn + 16 * n.value, r0 + wm, lane);
    wave_lds_fence();
  });
}

// ---------------------------------------------------------------------------
// joining the splits: y = the sum of the planes, in their order
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void vq_mx4_join_kernel(Mx4Args a, int splits) { join_planes(a, splits); }

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <int XK, int WAVES, int MT, int NL, int DEPTH>
void run_skinny(const Mx4Args& a, int, int splits, hipStream_t s) {
  constexpr int kTok = Mx4Slot<XK, 1, MT, NL>::kRows;
  const dim3 grid((unsigned)ceil_div(a.rows, 16 * MT) * ceil_div(a.T, kTok), splits);
  hipLaunchKernelGGL((vq_mx4_skinny_kernel<XK, WAVES, MT, NL, DEPTH>), grid, dim3(64 * WAVES), 0, s, a);
}

template <int WM, int WN, int MT, int NT, int KW>
void run_tile(const Mx4Args& a, int, int splits, hipStream_t s) {
  const dim3 grid((unsigned)ceil_div(a.rows, 16 * MT * WM) * ceil_div(a.T, 16 * NT * WN), splits);
  const dim3 block(64 * WM * WN * KW);
  if (a.y_kind == kOutF32) hipLaunchKernelGGL((vq_mx4_tile_kernel<true, WM, WN, MT, NT, KW>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((vq_mx4_tile_kernel<false, WM, WN, MT, NT, KW>), grid, block, 0, s, a);
}

template <int WM, int WN, int MT, int NT, int KW>
void run_tile16(const Mx4Args& a, int xk, int splits, hipStream_t s) {
  const dim3 grid((unsigned)ceil_div(a.rows, 16 * MT * WM) * ceil_div(a.T, 16 * NT * WN), splits);
  const dim3 block(64 * WM * WN * KW);
  auto run = [&](auto kind, auto precise) {
    hipLaunchKernelGGL((vq_mx4_tile16_kernel<decltype(kind)::value, decltype(precise)::value, WM, WN, MT, NT, KW>), grid,
                       block, 0, s, a);
  };
  const std::integral_constant<int, kMx4XF16> f16{};
  const std::integral_constant<int, kMx4XBF16> bf16{};
  if (a.y_kind == kOutF32) xk == kMx4XF16 ? run(f16, std::true_type{}) : run(bf16, std::true_type{});
  else xk == kMx4XF16 ? run(f16, std::false_type{}) : run(bf16, std::false_type{});
}

template <int WAVES, int MT, int NL, int DEPTH>
void run_skinny16(const Mx4Args& a, int xk, int splits, hipStream_t s) {
  if (xk == kMx4XF16) run_skinny<kMx4XF16, WAVES, MT, NL, DEPTH>(a, xk, splits, s);
  else run_skinny<kMx4XBF16, WAVES, MT, NL, DEPTH>(a, xk, splits, s);
}

// The kernels of the product and a time model of each (us), fitted to measured
// calls of 2152 shapes (1 to 4096 tokens, 16 to 17408 rows, 32 to 17408 columns,
// 1 to 24 splits), each with its weight in memory, as in a pass through a model's
// layers, and in the card's cache.  With weights from memory make_plan's choice
// takes 0.8 % longer than the shape's best call on average with 4-bit x and 0.5 %
// with 16-bit x (27 % at worst), on shapes kept apart 0.7 % (159, 38 %) and 1.7 %
// (419, 40 %); with cached weights 1.0 to 2.0 %.  The calls, the fit and the same
// choice replayed:
// profiles/mx4_product_calls.txt, profiles/mx4_plan_fit.py.
//   base + 4-norm(latency * steps, rounds * (rate * steps + unit), bytes / bw)
//   and, split, kMx4Split + join * (bytes of the planes, written and read, in MB)
// with steps of 128 columns a wave runs through, rounds of 256 blocks, and
// bytes the weight once, y, and the tokens once and `x_share` of that for every
// further row tile (MB; bw in TB/s).  The constants are fitted to the order of the
// calls first: predicted times are off by about a fifth.  Past the fitted sizes (up
// to 100000 tokens, 65536 rows and columns, 33 shapes) the choice is within 10 %.
struct Mx4Kernel {
  int rows, tokens;  // of a block
  int k_waves;       // waves, or groups of them, that split a block's columns
  int unit_blocks;   // splits are multiples of these blocks of columns
  bool mx4;          // 4-bit x (else 16-bit)
  float base, latency, rate, bw, join, unit, x_share;
  void (*run)(const Mx4Args&, int, int, hipStream_t);
};
const Mx4Kernel kMx4Kernels[] = {
    // 4-bit x: streams for few tokens, then tiles, with groups of waves where there are few
    {16, 8, 4, 8, true, 0.0721f, 0.209f, 0.102f, 12, 0.635f, 0.844f, 3.26f, run_skinny<kMx4XMx4, 4, 1, 1, 2>},
    {16, 16, 4, 8, true, 0.464f, 0.174f, 0.176f, 10.9f, 0.255f, 0.697f, 2.22f, run_skinny<kMx4XMx4, 4, 1, 2, 2>},
    {32, 16, 4, 8, true, 1.17f, 0.0388f, 0.222f, 10.8f, 0.423f, 1.06f, 3.75f, run_skinny<kMx4XMx4, 4, 2, 2, 2>},
    {128, 32, 1, 16, true, 0.0073f, 0.549f, 0.147f, 6.49f, 0.371f, 1.48f, 2.24f, run_tile<4, 1, 2, 2, 1>},
    {128, 32, 2, 32, true, 1.39f, 0.00304f, 0.628f, 12, 0.0332f, 3.08f, 0.166f, run_tile<4, 1, 2, 2, 2>},
    {128, 64, 2, 32, true, 0.129f, 0.00284f, 0.553f, 11.5f, 0.244f, 6.82f, 0.252f, run_tile<4, 1, 2, 4, 2>},
    {64, 32, 4, 64, true, 0.029f, 0.00854f, 0.609f, 12, 0.00328f, 4.83f, 0.118f, run_tile<2, 1, 2, 2, 4>},
    {64, 64, 2, 32, true, 0.364f, 0.491f, 0.192f, 12, 0.00643f, 8.91f, 0.073f, run_tile<2, 1, 2, 4, 2>},
    {128, 128, 1, 16, true, 6.01f, 0.0773f, 0.394f, 12, 0.183f, 0.017f, 0.0517f, run_tile<4, 2, 2, 4, 1>},
    {256, 128, 1, 16, true, 0.709f, 0, 0.531f, 12, 0.106f, 12, 0.292f, run_tile<4, 2, 4, 4, 1>},
    {256, 192, 1, 16, true, 8.08f, 0.002f, 0.55f, 12, 0.112f, 11.8f, 0.234f, run_tile<4, 2, 4, 6, 1>},
    {256, 256, 1, 16, true, 9.15f, 0.002f, 0.772f, 12, 0.131f, 9.17f, 0.216f, run_tile<4, 2, 4, 8, 1>},
    // 16-bit x: the same
    {16, 2, 4, 8, false, 0, 0.229f, 0.0164f, 12, 12, 1.28f, 8.17f, run_skinny16<4, 1, 1, 2>},
    {16, 4, 4, 8, false, 0.919f, 0.237f, 0.17f, 10.2f, 0.403f, 0.799f, 0, run_skinny16<4, 1, 2, 2>},
    {16, 8, 4, 8, false, 0.868f, 0.266f, 0.218f, 4.19f, 0.0251f, 0.997f, 0.176f, run_skinny16<4, 1, 4, 2>},
    {32, 16, 4, 8, false, 3.77f, 0.274f, 0.474f, 7.36f, 0.244f, 0.915f, 0.0191f, run_skinny16<4, 2, 8, 2>},
    {32, 16, 8, 8, false, 0, 0.00811f, 1.08f, 11.3f, 3.41f, 2.61f, 0, run_skinny16<8, 2, 8, 1>},
    {64, 16, 4, 16, false, 0, 0.0117f, 1.04f, 12, 0.00273f, 1.96f, 0, run_tile16<2, 1, 2, 1, 4>},
    {64, 32, 4, 16, false, 0, 0.0161f, 1.1f, 6.46f, 0.15f, 3.68f, 0.992f, run_tile16<2, 1, 2, 2, 4>},
    {64, 32, 2, 8, false, 1.84f, 0.943f, 0.427f, 3.64f, 0.133f, 1.66f, 0.125f, run_tile16<2, 1, 2, 2, 2>},
    {128, 32, 2, 8, false, 0, 0.978f, 0.667f, 12, 0.376f, 4.07f, 0, run_tile16<4, 1, 2, 2, 2>},
    {128, 64, 2, 8, false, 0, 0.015f, 1.1f, 12, 0, 8.47f, 0, run_tile16<4, 1, 2, 4, 2>},
    {128, 64, 1, 4, false, 3.57f, 0.765f, 0.571f, 6.44f, 0.253f, 0.0119f, 0.0237f, run_tile16<4, 2, 2, 2, 1>},
    {256, 128, 1, 4, false, 2.36f, 0.0247f, 1.36f, 12, 0.0988f, 12, 0, run_tile16<4, 2, 4, 4, 1>},
};
constexpr int kNumMx4Kernels = sizeof(kMx4Kernels) / sizeof(kMx4Kernels[0]);
constexpr float kMx4Split = 3.83f;  // us of the launch that joins a split's planes
constexpr int kMx4Splits[] = {1, 2, 3, 4, 6, 8, 12};  // (16 and 24 were the best of no fitted shape)
constexpr size_t kMaxPlanBytes = (size_t)512 << 20;  // planes of a split

// Sizes a plan is for.
struct Mx4Call {
  int rows, blocks, T;
  bool mx4;
  bool operator==(const Mx4Call& o) const {
    return rows == o.rows && blocks == o.blocks && T == o.T && mx4 == o.mx4;
  }
};

// The call by kernel i with its columns in up to `splits` parts.  False where
// the kernel does not serve the call, or the launch (fewer than 2^32 threads, a
// block up to 512) or the planes grow too large.
bool set_plan(const Mx4Call& c, int i, int splits, Mx4Plan* p) {
  const Mx4Kernel& k = kMx4Kernels[i];
  if (k.mx4 != c.mx4) return false;
  if ((int64_t)ceil_div(c.rows, k.rows) * ceil_div(c.T, k.tokens) >= 1 << 22) return false;
  p->kernel = i;
  p->split_blocks = ceil_div(ceil_div(c.blocks, splits), k.unit_blocks) * k.unit_blocks;
  p->splits = ceil_div(c.blocks, p->split_blocks);
  p->workspace = p->splits > 1 ? (size_t)p->splits * c.T * c.rows * sizeof(float) : 0;
  return p->workspace <= kMaxPlanBytes;
}

float plan_time(const Mx4Call& c, const Mx4Plan& p) {
  const Mx4Kernel& k = kMx4Kernels[p.kernel];
  const int row_tiles = ceil_div(c.rows, k.rows);
  const float split_steps = 0.25f * p.split_blocks, load_steps = split_steps / k.k_waves;
  const int64_t units = (int64_t)row_tiles * ceil_div(c.T, k.tokens) * p.splits;
  const float out = (float)c.T * c.rows, w = 17.0f * c.rows * c.blocks, x = (c.mx4 ? 17.0f : 64.0f) * c.T * c.blocks;
  const float bytes = (w + 4.0f * out + (1.0f + k.x_share * (row_tiles - 1)) * x) * 1e-6f;
  const float a = k.latency * std::ceil(load_steps), b = (float)((units + 255) / 256) * (k.rate * load_steps + k.unit),
              e = bytes / k.bw;
  const float t = k.base + std::sqrt(std::sqrt(a * a * a * a + b * b * b * b + e * e * e * e));
  return p.splits > 1 ? t + kMx4Split + k.join * p.splits * out * 8e-6f : t;
}

Mx4Plan make_plan(const Mx4Call& c) {
  Mx4Plan best;
  float best_t = 0.0f;
  for (int i = 0; i < kNumMx4Kernels; ++i) {
    for (const int s : kMx4Splits) {
      Mx4Plan p;
      if (!set_plan(c, i, s, &p) || p.splits != s) continue;
      const float t = plan_time(c, p);
      if (best.kernel < 0 || t < best_t) best = p, best_t = t;
    }
  }
  return best;
}

Mx4Plan cached_plan(const Mx4Call& c) {
  // the plans this thread made last (choosing takes a microsecond or two)
  struct Slot {
    Mx4Call call{};  // no rows: empty
    Mx4Plan plan;
  };
  static thread_local Slot last[64];
  Slot& slot = last[((unsigned)c.rows * 31u + (unsigned)c.blocks * 7u + (unsigned)c.T * 2u + (unsigned)c.mx4) % 64u];
  if (!(slot.call == c)) slot.plan = make_plan(c), slot.call = c;
  return slot.plan;
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

// VQMI_MX4_PLAN = "kernel,splits" (a row of the table) forces the choice, for
// tests; a kernel or split that set_plan refuses is passed over.
Mx4Plans mx4_plans(int rows, int cols, int T) {
  const char* e = getenv("VQMI_MX4_PLAN");
  int k = 0, splits = 0;
  const bool forced = e && sscanf(e, "%d,%d", &k, &splits) == 2 && k >= 0 && k < kNumMx4Kernels && splits >= 1 &&
                      splits <= 64;
  auto plan = [&](bool mx4) {
    const Mx4Call c{rows, cols / kMx4Block, T, mx4};
    Mx4Plan p;
    return forced && set_plan(c, k, splits, &p) ? p : cached_plan(c);
  };
  return {plan(true), plan(false)};
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
  a.part = p.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  a.split_blocks = p.split_blocks;
  kMx4Kernels[p.kernel].run(a, x_kind, p.splits, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const dim3 grid((unsigned)ceil_div((int64_t)T * w.rows, 1024));
  hipLaunchKernelGGL(vq_mx4_join_kernel, grid, dim3(256), 0, s, a, p.splits);
  return hipGetLastError();
}

}  // namespace vqmi
