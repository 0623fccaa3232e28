// vq_fp8.hip -- tensors in e4m3 with a scale for each block of 128: the
// quantizer of activations and the product of two such tensors.
//
//   quantize  s[t][b] = fl32(max |x| over the block / 448), q = e4m3(x / s)
//   product   y[t][r] = sum_b s_x[t][b] * s_w[r / 128][b] * sum_{c in b} x[t][c] * w[r][c]
//
// The times below are those of calls replayed from a graph over weights that
// do not stay in the caches, on a card that copies at 5.06 TB/s and reaches
// 3.2 PFLOP/s in the library's e4m3 product of 8192 x 8192 x 8192.
#include "vq_block_device.h"
#include "vq_fp8_device.h"
#include "vq_block_kernels.h"
#include "vq_store_device.h"

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <type_traits>

namespace vqmi {

namespace {

// ---------------------------------------------------------------------------
// quantizer: 16 lanes per block of 128 columns, 8 values each
//
// Bound by its bytes: two read, one written and a scale per 128.  16 lanes of
// 16 bytes make a block's maximum a matter of four DPP steps, no LDS, and its
// loads and stores whole lines; the maximum is taken from the 16-bit patterns.
// 4096 x 5120 in 14.8 to 15.3 us = 4.1 to 4.2 TB/s (13.2 where the input is still in the
// caches), 4 x 17408 in 2.3 us, a launch.
// ---------------------------------------------------------------------------
template <bool BF16>
__global__ __launch_bounds__(256) void vq_fp8_quant_kernel(const uint16_t* x, uint8_t* q, float* scales, uint32_t T,
                                                           uint32_t cols, uint32_t kb) {
  const uint32_t b = blockIdx.x * 16u + (threadIdx.x >> 4);  // block of 128 columns, row by row
  const uint32_t t = b / kb, k = b - t * kb;
  const uint32_t c = k * kFp8Block + (threadIdx.x & 15u) * 8u;
  const bool in = t < T && c < cols;  // cols is a multiple of 16
  const int64_t at = (int64_t)t * cols + c;
  u32x4 raw = {0u, 0u, 0u, 0u};
  if (in) raw = *reinterpret_cast<const u32x4*>(x + at);
  // the largest magnitude from the 16-bit patterns, two at a time
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m2 = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) m2 = __builtin_elementwise_max(m2, __builtin_bit_cast(u16x2, raw[i] & 0x7fff7fffu));
  const uint32_t m = max((uint32_t)m2.x, (uint32_t)m2.y);
  const uint32_t top = BF16 ? m << 16 : __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)m));
  float v[8], s;
  unpack8<BF16>(raw, v);
  const u32x2 codes = fp8_quantize8(v, top, &s);
  if (in) *reinterpret_cast<u32x2*>(q + at) = codes;
  if (t < T && (threadIdx.x & 15u) == 0) scales[b] = s;
}

// ---------------------------------------------------------------------------
// product, few tokens: a block takes 16 rows of w and 16 to 64 tokens, its
// waves split the blocks of 128 columns and join their sums in LDS
//
// Bound by the weights' bytes.  Blocks of 16 rows are enough of them to fill
// the card at 5120 rows already.  With 16 tokens a block takes four waves with
// two column blocks in flight each (64 registers: every block of 17408 rows is
// on the card at once), with 32 or 64 eight waves with one.  One token, 17408 x
// 5120: 22 us = 4.1 TB/s (18 in a plain stream of calls on the same weights),
// 34816 x 5120: 37.  At 16, eight waves took 22.5 and 39, five column blocks in
// flight 24, and 16 waves a block or columns that start elsewhere in every
// block were no faster.  From a few tokens on a 128 x 32 tile with the columns
// split may be faster (16 tokens, 5120 x 17408: 24.4 against 31), and few rows
// with many tokens may do better here (991 tokens, 29 rows: 6.9 against 12.5).
// ---------------------------------------------------------------------------
struct Fp8Args {
  const uint8_t* w;
  const float* ws;
  const uint8_t* x;
  const float* xs;
  void* y;
  int rows, cols, kb, T;
  int y_kind, swiglu;
  float* part;      // split columns: fp32 sums [gridDim.y][T][rows] in place of y
  int split_steps;  // column blocks a split (the last one may have fewer)
};

// The arguments of one split of the columns: its sums go to their own plane of
// the workspace, as they are.
__device__ __forceinline__ Fp8Args split_args(Fp8Args a) {
  if (a.part) {
    a.y = a.part + (int64_t)blockIdx.y * a.T * a.rows;
    a.y_kind = kOutF32;
    a.swiglu = 0;
  }
  return a;
}

// A lane's 32 bytes of 16 rows x 128 columns (row = lane % 16): columns
// 16 * (lane / 16) .. + 15 and the same behind column 64.  Both operands are
// taken this way, so the columns meet their own; pieces past the last column
// (or row: past the buffer) read as zeros.
struct Frag {
  u32x4 lo, hi;
};
__device__ __forceinline__ Frag load_frag(rsrc_t r, uint32_t row_off, uint32_t c, uint32_t cols) {
  return {buf_load_b128(r, c < cols ? row_off + c : kOutOfRange),
          buf_load_b128(r, c + 64 < cols ? row_off + c + 64 : kOutOfRange)};
}

// Eight e4m3 codes as halves, exactly.
__device__ __forceinline__ half8_t to_half8(uint32_t w0, uint32_t w1) {
  const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, false);
  const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, true);
  const half2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, false);
  const half2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, true);
  return half8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// The sums of 128 products of 16 x 16 outputs through fp16 operands.  An e4m3
// value is an fp16 value, and the fp16 matrix instructions sum exact products
// in fp32.  The e4m3 ones cut every product of a group of eight 13 bits below
// the group's largest (measured: a 2-norm error of 1.6e-5 on normal inputs
// against 8e-9 here), so where large products cancel small ones are lost:
// they serve only calls that ask for them.
__device__ __forceinline__ float4_t dot128_f16(const Frag& a, const Frag& b) {
  float4_t p = {0.0f, 0.0f, 0.0f, 0.0f};
  p = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_half8(a.lo.x, a.lo.y), to_half8(b.lo.x, b.lo.y), p, 0, 0, 0);
  p = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_half8(a.lo.z, a.lo.w), to_half8(b.lo.z, b.lo.w), p, 0, 0, 0);
  p = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_half8(a.hi.x, a.hi.y), to_half8(b.hi.x, b.hi.y), p, 0, 0, 0);
  p = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_half8(a.hi.z, a.hi.w), to_half8(b.hi.z, b.hi.w), p, 0, 0, 0);
  return p;
}

// NT x 16 tokens a block; a wave takes every WAVES-th block of 128 columns and
// has DEPTH of them in flight.  The products of the scales of a chunk of
// kChunk column blocks are set up in LDS first, so the loop waits for
// nothing but its operands.
constexpr int kScaleSteps = 256;

template <int WAVES, int NT, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void vq_fp8_skinny_kernel(Fp8Args args) {
  const Fp8Args a = split_args(args);
  constexpr int kThreads = 64 * WAVES, kTok = 16 * NT;
  constexpr int kChunk = kScaleSteps / NT;  // column blocks per chunk: 16 KiB of scales
  __shared__ float f[kChunk][kTok];
  __shared__ float4_t part[WAVES][NT][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const unsigned row_tiles = (a.rows + 15) / 16;  // row tiles run fastest: they share the tokens
  const int r0 = (blockIdx.x % row_tiles) * 16, t0 = (blockIdx.x / row_tiles) * kTok;
  const int r = lane & 15;
  const uint32_t cols = a.cols;
  const int kb = a.kb;
  const rsrc_t wr = make_rsrc(a.w + (int64_t)r0 * cols, (uint64_t)min(16, a.rows - r0) * cols);
  const rsrc_t xr = make_rsrc(a.x + (int64_t)t0 * cols, (uint64_t)min(kTok, a.T - t0) * cols);
  const rsrc_t sr = make_rsrc(a.xs + (int64_t)t0 * kb, (uint64_t)min(kTok, a.T - t0) * kb * 4);
  const rsrc_t wsr = make_rsrc(a.ws + (int64_t)(r0 / kFp8Block) * kb, (uint64_t)kb * 4);
  float4_t acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  Frag aw[DEPTH], bx[DEPTH][NT];
  auto load = [&](int j, int k) {  // steps past the end: zeros
    const uint32_t c = k * kFp8Block + (lane >> 4) * 16;
    aw[j] = load_frag(wr, r * cols, c, cols);
#pragma unroll
    for (int n = 0; n < NT; ++n) bx[j][n] = load_frag(xr, (16 * n + r) * cols, c, cols);
  };
  const int k_first = blockIdx.y * a.split_steps, k_end = min(kb, k_first + a.split_steps);
  for (int k0 = k_first; k0 < k_end; k0 += kChunk) {
    const int steps = min(kChunk, k_end - k0);
    if (k0 > k_first) __syncthreads();
    // a thread's scale products: token-major reads (the steps of a token lie
    // side by side), step-major in LDS
    constexpr int kPer = kChunk * kTok / kThreads;
    float sx[kPer], sw[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = threadIdx.x + i * kThreads, t = e / kChunk, k = e % kChunk;
      const uint32_t ok = k < steps ? 0u : kOutOfRange;
      sx[i] = __uint_as_float(buf_load_b32(sr, ok | (uint32_t)(t * kb + k0 + k) * 4));
      sw[i] = __uint_as_float(buf_load_b32(wsr, ok | (uint32_t)(k0 + k) * 4));
    }
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) load(j, wave + j * WAVES < steps ? k0 + wave + j * WAVES : kb);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = threadIdx.x + i * kThreads;
      f[e % kChunk][e / kChunk] = sx[i] * sw[i];
    }
    lds_barrier();
    for (int k = wave; k < steps; k += DEPTH * WAVES) {
#pragma unroll
      for (int j = 0; j < DEPTH; ++j) {
        // no branches: the loads in flight are counted through the loop
        const int kj = k + j * WAVES, next = kj + DEPTH * WAVES;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float4_t p = dot128_f16(aw[j], bx[j][n]);
          const float s = DEPTH == 1 || kj < steps ? f[min(kj, kChunk - 1)][16 * n + r] : 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][i] = fmaf(s, p[i], acc[n][i]);
        }
        load(j, next < steps ? k0 + next : kb);
      }
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
  if (t < a.T) store_rows4(a, t, r0 + (lane >> 4) * 4, v);
}

// ---------------------------------------------------------------------------
// product, many tokens: WM x WN waves of 16*MT rows x 16*NT tokens a block
//
// The scales change with every 128 columns, so a product of 16 x 16 x 128 is
// one instruction and four FMAs a lane scale it into the sums.  Of a 256 x 192
// step the e4m3 instructions are 1536 cycles at their peak, 1940 with the FMAs
// and addresses; LDS is busy for 1400 (reads at 249 bytes a cycle, writes at
// 80), and a block alone takes 2360.  With every compute unit busy the clock
// falls to 1.85 GHz: what moves fewer bytes for a product gains twice.
//   - 8 waves (two a SIMD: one's FMAs and LDS reads run under the other's
//     products) take 212 us where 4 waves of 128 x 96 took 245;
//   - operands are read two products ahead, sums scaled two products behind
//     (212 -> 202), across steps;
//   - global loads pass through registers into LDS, spread over the step:
//     with loads straight to LDS the compiler waits for all of them before
//     the next LDS read;
//   - one barrier a step, two buffers, pieces XORed so that reads of 8 rows
//     touch all banks.
// 2048 tokens x 17408 x 5120 in bf16: 182 to 201 us on different cards, 1.8 to
// 2.0 PFLOP/s, with SwiGLU (half the outputs) the same; 4096 x 8192 x 8192: 230
// to 249 us, 2.2 to 2.4 PFLOP/s.  Those are the e4m3 instructions
// (vq_fp8_gemm_fast).  Exact products cost four fp16 instructions of 16 cycles
// for one e4m3 of 32, and their conversions: 370 to 384 us there for any y, and
// 499 at 4096 x 8192 x 8192 (1.0 and 1.1 PFLOP/s).
// ---------------------------------------------------------------------------
typedef int int8v __attribute__((ext_vector_type(8)));

// One operand of the 16 x 16 x 128 products: e4m3 as it is, or (EXACT) as halves.
template <bool EXACT>
struct Op {
  int8v v;
  __device__ __forceinline__ void set(u32x4 lo, u32x4 hi) {
    v = int8v{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  }
};
template <>
struct Op<true> {
  half8_t v[4];
  __device__ __forceinline__ void set(u32x4 lo, u32x4 hi) {
    v[0] = to_half8(lo.x, lo.y);
    v[1] = to_half8(lo.z, lo.w);
    v[2] = to_half8(hi.x, hi.y);
    v[3] = to_half8(hi.z, hi.w);
  }
};
template <bool EXACT>
__device__ __forceinline__ float4_t dot128(const Op<EXACT>& a, const Op<EXACT>& b) {
  float4_t p = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (EXACT) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[i], b.v[i], p, 0, 0, 0);
  } else {
    p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, p, 0, 0, 0, 0, 0, 0);
  }
  return p;
}

template <bool EXACT, int WM, int WN, int MT, int NT, int AHEAD>
__global__ __launch_bounds__(64 * WM * WN, WM * WN / 4) void vq_fp8_tile_kernel(Fp8Args args) {
  const Fp8Args a = split_args(args);
  constexpr int kWaves = WM * WN, kTileRows = 16 * MT * WM, kTileTokens = 16 * NT * WN;
  constexpr int kLoadRows = 8 * kWaves;  // rows the block loads at once
  constexpr int kWLoads = kTileRows / kLoadRows, kXLoads = kTileTokens / kLoadRows, kLoads = kWLoads + kXLoads;
  static_assert(kTileRows % kLoadRows == 0 && kTileTokens % kLoadRows == 0, "whole loads");
  static_assert(128 % (16 * MT) == 0, "a wave's rows share their scales");
  static_assert(kTileTokens <= 256 && NT % (AHEAD + 1) == 0, "scales of at most 256 tokens; a ring of operands");
  __shared__ __align__(1024) uint8_t lds_w[2][kTileRows * 128];
  __shared__ __align__(1024) uint8_t lds_x[2][kTileTokens * 128];
  __shared__ __align__(1024) float lds_s[2][256][4];  // x scales of four steps, twice
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t cols = a.cols, kb = a.kb;

  const int row_tiles = (a.rows + kTileRows - 1) / kTileRows, tok_tiles = (a.T + kTileTokens - 1) / kTileTokens;
  int rt, tt;
  xcd_tile(blockIdx.x, row_tiles, tok_tiles, &rt, &tt);
  const int r0 = rt * kTileRows, t0 = tt * kTileTokens;
  const rsrc_t wr = make_rsrc(a.w + (int64_t)r0 * cols, (uint64_t)min(kTileRows, a.rows - r0) * cols);
  const rsrc_t xr = make_rsrc(a.x + (int64_t)t0 * cols, (uint64_t)min(kTileTokens, a.T - t0) * cols);
  const rsrc_t sr = make_rsrc(a.xs + (int64_t)t0 * kb, (uint64_t)min(kTileTokens, a.T - t0) * kb * 4);
  const int wm = wave / WN * 16 * MT, wn = wave % WN * 16 * NT;  // the wave's rows and tokens
  // rows past the end multiply zeros: any block of scales will do
  const float* ws = a.ws + (int64_t)min((r0 + wm) / kFp8Block, (a.rows - 1) / kFp8Block) * kb;

  // A wave loads 8 rows of 128 bytes at a time, 16 bytes a lane, through
  // registers into LDS.  The 16-byte pieces of row r lie in the order piece ^
  // (r % 8), so the fragment reads of 8 rows touch all banks.  Columns, rows
  // and steps past the end arrive as zeros.
  const uint32_t ld_piece = (lane & 7) * 16, ld_row = wave * 8 + (lane >> 3);
  const uint32_t ld_dst = ld_row * 128 + (ld_piece ^ ((lane >> 3) * 16));
  // steps of this split: s0 is a multiple of four
  const uint32_t s0 = blockIdx.y * a.split_steps, s1 = min(kb, s0 + a.split_steps);
  u32x4 stage[kLoads];
  float stage_s;
  auto stage_off = [&](uint32_t s) {
    const uint32_t c = s * kFp8Block + ld_piece;
    return s < s1 && c < cols ? ld_row * cols + c : kOutOfRange;
  };
  auto load_piece = [&](uint32_t off, int i) {
    stage[i] = i < kWLoads ? buf_load_b128(wr, off + i * kLoadRows * cols)
                           : buf_load_b128(xr, off + (i - kWLoads) * kLoadRows * cols);
  };
  auto write_piece = [&](uint32_t s, int i) {
    uint8_t* to = i < kWLoads ? lds_w[s & 1] + i * kLoadRows * 128 : lds_x[s & 1] + (i - kWLoads) * kLoadRows * 128;
    *reinterpret_cast<u32x4*>(to + ld_dst) = stage[i];
  };
  // Scales of the four steps from v & ~3 on, for the quarter v % 4 of the
  // tokens (four lanes a token; every four waves load the same).
  const uint32_t sc_tok = (wave & 3) * 16 + (lane >> 2);
  auto load_scales = [&](uint32_t v) {
    const uint32_t tok = (v & 3) * 64 + sc_tok, k = (v & ~3u) + (lane & 3);
    stage_s = __uint_as_float(buf_load_b32(sr, k < kb && tok < kTileTokens ? (tok * kb + k) * 4 : kOutOfRange));
  };
  auto write_scales = [&](uint32_t v) { lds_s[(v >> 2) & 1][(v & 3) * 64 + sc_tok][lane & 3] = stage_s; };
  const int r = lane & 15, g = lane >> 4;
  const uint32_t f_lo = r * 128 + ((g ^ (r & 7)) * 16), f_hi = r * 128 + (((g + 4) ^ (r & 7)) * 16);
  auto read_op = [&](Op<EXACT>& o, const uint8_t* base) {
    o.set(*reinterpret_cast<const u32x4*>(base + f_lo), *reinterpret_cast<const u32x4*>(base + f_hi));
  };

  float4_t acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // The first step with the scales of its group (and a quarter of the next) in
  // LDS, the second in registers.
#pragma unroll
  for (uint32_t v = 0; v < 5; ++v) {
    load_scales(s0 + v);
    write_scales(s0 + v);
  }
#pragma unroll
  for (uint32_t s = 0; s < 2; ++s) {
    const uint32_t off = stage_off(s0 + s);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load_piece(off, i);
    if (s < 1) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) write_piece(s, i);
    }
  }
  load_scales(s0 + 5);
  lds_barrier();
  constexpr int kRing = AHEAD + 1;  // token operands: the current one and the next AHEAD
  Op<EXACT> av[MT], bv[kRing];
#pragma unroll
  for (int m = 0; m < MT; ++m) read_op(av[m], lds_w[0] + (wm + 16 * m) * 128);
#pragma unroll
  for (int n = 0; n < AHEAD; ++n) read_op(bv[n], lds_x[0] + (wn + n * 16) * 128);
  float f[NT], f_last = 0.0f;
#pragma unroll
  for (int n = 0; n < NT; ++n) f[n] = ws[s0] * lds_s[(s0 >> 2) & 1][wn + 16 * n + r][0];

  // The sums of two products stay in flight while the ones before them are
  // scaled into the accumulators, across steps too.
  constexpr int kLag = 2;
  float4_t p[kLag];
#pragma unroll
  for (int i = 0; i < kLag; ++i) p[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  for (uint32_t s = s0; s < s1; ++s) {
    const uint8_t* xb = lds_x[s & 1] + wn * 128;
    const uint8_t* xnext = lds_x[(s + 1) & 1] + wn * 128;
    const uint8_t* wnext = lds_w[(s + 1) & 1] + wm * 128;
    const float sw_next = ws[min(s + 1, kb - 1)];
    const uint32_t off = stage_off(s + 2);
    float f_next[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // every wave has issued its last reads of this step before the barrier
      // waits for them, so behind it the next step's pieces in LDS are complete
      // and this one's buffers free
      if (n == NT - AHEAD) lds_barrier();
      read_op(bv[(n + AHEAD) % kRing], (n + AHEAD < NT ? xb : xnext) + (n + AHEAD) % NT * 16 * 128);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int i = n * MT + m;
        const float4_t now = dot128<EXACT>(av[m], bv[n % kRing]);
        __builtin_amdgcn_sched_barrier(0);
        // the next step's pieces go to LDS, spread over the step, and the ones
        // after them are loaded in their place
        constexpr int kSlots = (NT - AHEAD) * MT;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          if (k * kSlots / kLoads == i) {
            write_piece(s + 1, k);
            load_piece(off, k);
          }
        }
        if (n == NT - 1) {
          read_op(av[m], wnext + m * 16 * 128);
#pragma unroll
          for (int k = m; k < NT; k += MT) f_next[k] = lds_s[((s + 1) >> 2) & 1][wn + 16 * k + r][(s + 1) & 3];
          if (m == MT - 1) {
            write_scales(s + 5);
            load_scales(s + 6);
          }
        }
        {
          const int j = i - kLag, jn = j >= 0 ? j / MT : NT - 1, jm = j >= 0 ? j % MT : MT + j;
          const float fj = j >= 0 ? f[jn] : f_last;
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[jm][jn][c] = fmaf(fj, p[i % kLag][c], acc[jm][jn][c]);
        }
        p[i % kLag] = now;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    f_last = f[NT - 1];
#pragma unroll
    for (int n = 0; n < NT; ++n) f[n] = sw_next * f_next[n];
  }
#pragma unroll
  for (int i = 0; i < kLag; ++i) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      acc[MT - kLag + i][NT - 1][c] = fmaf(f_last, p[i][c], acc[MT - kLag + i][NT - 1][c]);
  }
  // The waves' outputs go through the same LDS, 16 tokens at a time, so that a
  // token's rows leave in whole pieces.
  lds_barrier();
  constexpr int kPitch = 16 * MT + 4;  // fp32 a token
  static_assert(kWaves * 16 * kPitch * 4 <= (int)sizeof(lds_w), "every wave's 16 tokens fit");
  float* out = reinterpret_cast<float*>(&lds_w[0][0]) + wave * 16 * kPitch;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int m = 0; m < MT; ++m) *reinterpret_cast<float4_t*>(out + r * kPitch + 16 * m + 4 * g) = acc[m][n];
    wave_lds_fence();
    store_tokens<16 * MT, EXACT>(a, out, kPitch, t0 + wn + 16 * n, r0 + wm, lane);
    wave_lds_fence();
  }
}

// ---------------------------------------------------------------------------
// joining the splits: y = the sum of the planes, in their order
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void vq_fp8_join_kernel(Fp8Args a, int splits) { join_planes(a, splits); }

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <bool EXACT, int WM, int WN, int MT, int NT, int AHEAD>
void run_tile(const Fp8Args& a, int splits, hipStream_t s) {
  const dim3 grid((unsigned)ceil_div(a.rows, 16 * MT * WM) * ceil_div(a.T, 16 * NT * WN), splits);
  hipLaunchKernelGGL((vq_fp8_tile_kernel<EXACT, WM, WN, MT, NT, AHEAD>), grid, dim3(64 * WM * WN), 0, s, a);
}

template <int WAVES, int NT, int DEPTH>
void run_skinny(const Fp8Args& a, int splits, hipStream_t s) {
  const dim3 grid((unsigned)ceil_div(a.rows, 16) * ceil_div(a.T, 16 * NT), splits);
  hipLaunchKernelGGL((vq_fp8_skinny_kernel<WAVES, NT, DEPTH>), grid, dim3(64 * WAVES), 0, s, a);
}

// The kernels of the product and a time model of each (us), fitted to 21180
// measured calls (1 to 4096 tokens, 32 to 34816 rows, 256 to 17408 columns, 1
// to 24 splits), the faster ones of a shape weighing more; the fit's error is
// 6-13 % rms.  The model's choice takes 1.7 % longer than the best one on
// average, 0.2 to 0.3 % for products of more than 100 us; exact products with
// a bf16 y, measured afterwards, 1.9 and 0.2 % (the calls and the fit:
// profiles/fp8_product_calls.txt, profiles/fp8_plan_fit.py):
//   base + 4-norm(latency * steps, rounds * (rate * steps + unit), bytes / bw)
//   and, split, 2 + join * (bytes of the planes, written and read, in MB)
// with steps the column blocks a wave runs through, rounds of 256 blocks, and
// bytes the weight once, y, and `x_share` of the tokens' reads by every row
// tile (MB; bw in TB/s).
struct Fp8Kernel {
  int rows, tokens;        // of a block
  int k_waves;             // waves that split a block's columns
  int min_T, max_T;        // tokens it is considered for
  bool exact, fast;        // calls it serves: exact products, e4m3 instructions allowed
  float base, latency, rate, bw, join, unit, x_share;
  void (*run)(const Fp8Args&, int, hipStream_t);
};
constexpr int kAnyT = 1 << 30;
const Fp8Kernel kFp8Kernels[] = {
    // columns split over a block's waves (fp16 instructions): few tokens or few rows
    {16, 16, 4, 1, kAnyT, true, true, 4.200f, 0.347f, 0.265f, 7.268f, 0.422f, 0.685f, 1.200f, run_skinny<4, 1, 2>},
    {16, 32, 8, 17, kAnyT, true, true, 4.055f, 1.362f, 0.648f, 7.871f, 0.241f, 1.700f, 1.200f, run_skinny<8, 2, 1>},
    {16, 64, 8, 17, kAnyT, true, true, 3.886f, 1.965f, 1.025f, 8.000f, 0.321f, 2.192f, 1.162f, run_skinny<8, 4, 1>},
    // tiles on fp16 instructions: exact products
    {128, 32, 1, 1, kAnyT, true, false, 4.034f, 0.682f, 0.349f, 5.276f, 0.169f, 1.087f, 0.650f,
     run_tile<true, 4, 1, 2, 2, 1>},
    {128, 64, 1, 1, kAnyT, true, false, 4.195f, 0.909f, 0.504f, 6.366f, 0.148f, 1.736f, 1.200f,
     run_tile<true, 4, 1, 2, 4, 1>},
    {128, 192, 1, 32, kAnyT, true, false, 5.953f, 1.008f, 1.368f, 3.543f, 0.181f, 1.149f, 0.665f,
     run_tile<true, 4, 2, 2, 6, 1>},
    {256, 128, 1, 32, kAnyT, true, false, 4.851f, 0.691f, 1.628f, 4.558f, 0.139f, 3.888f, 1.200f,
     run_tile<true, 4, 2, 4, 4, 1>},
    // tiles on e4m3 instructions
    {128, 32, 1, 1, kAnyT, false, true, 4.105f, 0.469f, 0.236f, 5.226f, 0.169f, 0.857f, 0.814f,
     run_tile<false, 4, 1, 2, 2, 1>},
    {128, 64, 1, 1, kAnyT, false, true, 4.169f, 0.510f, 0.300f, 5.329f, 0.155f, 1.299f, 0.674f,
     run_tile<false, 4, 1, 2, 4, 1>},
    {128, 192, 1, 32, kAnyT, false, true, 3.997f, 0.003f, 0.713f, 5.712f, 0.173f, 2.684f, 0.615f,
     run_tile<false, 4, 2, 2, 6, 1>},
    {256, 192, 1, 32, kAnyT, false, true, 6.537f, 0.000f, 1.026f, 6.435f, 0.151f, 2.174f, 1.200f,
     run_tile<false, 4, 2, 4, 6, 2>},
    {256, 256, 1, 32, kAnyT, false, true, 7.251f, 0.010f, 1.357f, 6.978f, 0.144f, 2.308f, 1.200f,
     run_tile<false, 4, 2, 4, 8, 1>},
};
constexpr int kNumFp8Kernels = sizeof(kFp8Kernels) / sizeof(kFp8Kernels[0]);
constexpr size_t kMaxPlanBytes = (size_t)512 << 20;  // planes of a split

// Sizes a plan is for.
struct Fp8Call {
  int rows, cols, T;
  bool fast;
  bool operator==(const Fp8Call& o) const {
    return rows == o.rows && cols == o.cols && T == o.T && fast == o.fast;
  }
};

// The call by kernel i with its columns in up to `splits` parts of whole column
// blocks (the tiles' groups of scales: whole fours).  False where the kernel
// does not serve the call, or the launch (fewer than 2^32 threads, a block up
// to 512) or the planes grow too large.
bool set_plan(const Fp8Call& c, int i, int splits, Fp8Plan* p) {
  const Fp8Kernel& k = kFp8Kernels[i];
  if (!(c.fast ? k.fast : k.exact)) return false;
  if ((int64_t)ceil_div(c.rows, k.rows) * ceil_div(c.T, k.tokens) >= 1 << 22) return false;
  const int kb = ceil_div(c.cols, kFp8Block), q = k.k_waves > 1 ? 1 : 4;
  p->kernel = i;
  p->split_steps = ceil_div(ceil_div(kb, splits), q) * q;
  p->splits = ceil_div(kb, p->split_steps);
  p->workspace = p->splits > 1 ? (size_t)p->splits * c.T * c.rows * sizeof(float) : 0;
  return p->workspace <= kMaxPlanBytes;
}

float plan_time(const Fp8Call& c, const Fp8Plan& p) {
  const Fp8Kernel& k = kFp8Kernels[p.kernel];
  const float steps = (float)ceil_div(p.split_steps, k.k_waves);
  const float load_steps = (float)p.split_steps / k.k_waves;
  const int64_t units = (int64_t)ceil_div(c.rows, k.rows) * ceil_div(c.T, k.tokens) * p.splits;
  const float out = (float)c.T * c.rows;
  const float bytes = ((float)c.rows * c.cols + 4.0f * out + k.x_share * (float)c.T * c.cols * c.rows / k.rows) * 1e-6f;
  const float a = k.latency * steps, b = (float)((units + 255) / 256) * (k.rate * load_steps + k.unit), e = bytes / k.bw;
  const float t = k.base + std::sqrt(std::sqrt(a * a * a * a + b * b * b * b + e * e * e * e));
  return p.splits > 1 ? t + 2.0f + k.join * p.splits * out * 8e-6f : t;
}

Fp8Plan make_plan(const Fp8Call& c) {
  Fp8Plan best;
  float best_t = 0.0f;
  for (int i = 0; i < kNumFp8Kernels; ++i) {
    if (c.T < kFp8Kernels[i].min_T || c.T > kFp8Kernels[i].max_T) continue;
    for (int s : {1, 2, 3, 4, 6, 8, 12, 16, 24}) {
      Fp8Plan p;
      if (!set_plan(c, i, s, &p) || p.splits != s) continue;
      const float t = plan_time(c, p);
      if (best.kernel < 0 || t < best_t) best = p, best_t = t;
    }
  }
  return best;
}

Fp8Plan cached_plan(const Fp8Call& c) {
  // the plans this thread made last (choosing takes a microsecond or two)
  struct Slot {
    Fp8Call call{};  // no rows: empty
    Fp8Plan plan;
  };
  static thread_local Slot last[64];
  Slot& slot = last[((unsigned)c.rows * 31u + (unsigned)c.cols * 7u + (unsigned)c.T * 2u + (unsigned)c.fast) % 64u];
  if (!(slot.call == c)) slot.plan = make_plan(c), slot.call = c;
  return slot.plan;
}

}  // namespace

hipError_t launch_fp8_quant(const void* x, int x_bf16, int T, int cols, uint8_t* q, float* scales, hipStream_t s) {
  const uint32_t kb = (uint32_t)(cols + kFp8Block - 1) / kFp8Block;
  const dim3 grid(((uint32_t)T * kb + 15u) / 16u), block(256);
  const uint16_t* xh = static_cast<const uint16_t*>(x);
  if (x_bf16) hipLaunchKernelGGL((vq_fp8_quant_kernel<true>), grid, block, 0, s, xh, q, scales, T, cols, kb);
  else hipLaunchKernelGGL((vq_fp8_quant_kernel<false>), grid, block, 0, s, xh, q, scales, T, cols, kb);
  return hipGetLastError();
}

// VQMI_FP8_PLAN = "kernel,splits" (a row of the table) forces the choice, for
// tests; a kernel or split that set_plan refuses is passed over.
Fp8Plans fp8_plans(int rows, int cols, int T) {
  const char* e = getenv("VQMI_FP8_PLAN");
  int k = 0, splits = 0;
  const bool forced = e && sscanf(e, "%d,%d", &k, &splits) == 2 && k >= 0 && k < kNumFp8Kernels && splits >= 1 &&
                      splits <= 64;
  auto plan = [&](bool fast) {
    const Fp8Call c{rows, cols, T, fast};
    Fp8Plan p;
    return forced && set_plan(c, k, splits, &p) ? p : cached_plan(c);
  };
  return {plan(false), plan(true)};
}

hipError_t launch_fp8_gemm(const Fp8View& w, const IoSpec& io, const Fp8Plan& p, const uint8_t* x, const float* xs,
                           int T, void* y, void* workspace, hipStream_t s) {
  Fp8Args a{};
  a.w = w.values;
  a.ws = w.scales;
  a.x = x;
  a.xs = xs;
  a.y = y;
  a.rows = w.rows;
  a.cols = w.cols;
  a.kb = ceil_div(w.cols, kFp8Block);
  a.T = T;
  a.y_kind = io.y_kind;
  a.swiglu = io.epi == kEpiSwiglu;
  a.part = p.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  a.split_steps = p.split_steps;
  kFp8Kernels[p.kernel].run(a, p.splits, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  hipLaunchKernelGGL(vq_fp8_join_kernel, dim3((unsigned)ceil_div((int64_t)T * w.rows, 1024)), dim3(256), 0, s, a,
                     p.splits);
  return hipGetLastError();
}

}  // namespace vqmi
