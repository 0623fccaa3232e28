// vq_norm.hip -- the norms before and after a block, fused with its gate and
// the scaled residual sum, and with the quantization of the next input.
//
//   u = block * rsqrt(mean(block^2) + eps) * (post_weight + offset)   (or block as it is)
//   v = beta * residual + alpha * act(gate) * u
//   h = v * rsqrt(mean(v^2) + eps) * (pre_weight + offset)
//
// The row stays in registers between its one read and its writes: 8 to 32
// values a thread, a wave to 16 waves a row.  All arithmetic and both
// sums of squares are fp32; v and h are rounded once, on their stores (h
// comes from the unrounded v).
//
// Bound by its bytes: 4096 x 5120 in bf16, both norms, v and h stored, takes
// 36 to 38 us = 4.4 to 4.7 TB/s, where a plain copy reaches 5.06; 333 x 2000 to
// e4m3 5.3, one token of 5120 4.5, twice a launch.  A row a block, without a
// loop over rows: persistent blocks with the next row in flight and the weights
// held took 63 to 98, as the registers cost more rows in flight than that put
// back.
#include "vq_fp8_device.h"
#include "vq_block_kernels.h"

namespace vqmi {

namespace {

struct NormArgs {
  const void* block;      // nullptr: none
  const void* residual;   // nullptr: none
  const void* post_w;     // nullptr: block as it is
  const void* pre_w;      // nullptr: factor 1
  const void* gate;
  void* v_out;            // nullptr: not stored
  void* h;                // nullptr: not computed
  float* h_scales;        // e4m3 h
  int T, cols, kb;
  int block_kind, res_kind, w_kind, h_kind;  // OutKind; h: kNormE4m3 too
  int gate_kind, gate_act;
  float alpha, beta, eps, offset, inv_cols;
};

// Eight values as they lie in memory: 32 bytes of fp32 (WIDE) or 16 of fp16 or
// bf16.
template <bool WIDE>
struct Raw8 {
  u32x4 q[WIDE ? 2 : 1];
};

template <bool WIDE>
__device__ __forceinline__ void to_float(const Raw8<WIDE>& r, int kind, float* x) {
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r.q[i / 4][i % 4]);
  } else if (kind == kOutF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = r.q[0][i];
      const half2_t h = __builtin_bit_cast(half2_t, w);
      x[2 * i] = (float)h.x;
      x[2 * i + 1] = (float)h.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(r.q[0][i] << 16);
      x[2 * i + 1] = __uint_as_float(r.q[0][i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ float load1(const void* p, int64_t i, int kind) {
  if (kind == kOutF32) return static_cast<const float*>(p)[i];
  if (kind == kOutF16) return (float)static_cast<const _Float16*>(p)[i];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

__device__ __forceinline__ void store8(void* p, int64_t i, const float* x, int kind) {
  if (kind == kOutF32) {
    u32x4* q = reinterpret_cast<u32x4*>(static_cast<float*>(p) + i);
    q[0] = u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
    q[1] = u32x4{__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])};
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = pack16(x[2 * k], x[2 * k + 1], kind == kOutF16);
  *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = u32x4{w[0], w[1], w[2], w[3]};
}

// exp(x) within two units: the product's rounding error goes into the result.
__device__ __forceinline__ float exp_near(float x) {
  const float t = x * 1.44269504f, lo = fmaf(x, 1.44269504f, -t) + x * 1.925963033e-8f;
  const float e = __builtin_amdgcn_exp2f(t);
  return e < INFINITY && e > 0.0f ? fmaf(e, lo * 0.693147181f, e) : e;
}

__device__ __forceinline__ float gate_act(float g, int act) {
  if (act == kGateSigmoid) return 1.0f / (1.0f + exp_near(-g));
  if (act == kGateTanh) {
    // near zero the odd series to x^11 (the rest below 2^-28 at 0.3)
    const float a = fabsf(g), q = g * g;
    float p = fmaf(q, -8.8632355e-3f, 2.1869489e-2f);
    p = fmaf(q, p, -5.3968254e-2f);
    p = fmaf(q, p, 1.3333333e-1f);
    p = fmaf(q, p, -3.3333333e-1f);
    const float small = fmaf(g * q, p, g), big = copysignf(1.0f - 2.0f / (1.0f + exp_near(2.0f * a)), g);
    return a < 0.3f ? small : (a >= 0.3f ? big : g);  // NaN stays
  }
  return g;
}

// Chunk c of a thread's row.  VEC 8: runs of 8 columns, 16-byte loads (cols a
// multiple of 8).  VEC 1: any cols, one column at a time, converted as loaded.
template <int VEC>
struct RowMap {
  int tid, threads, cols;  // threads: of a row
  __device__ __forceinline__ int col(int c, int j) const {
    return VEC == 8 ? (c * threads + tid) * 8 + j : (c * 8 + j) * threads + tid;
  }
  __device__ __forceinline__ bool in(int c, int j) const { return col(c, VEC == 8 ? 0 : j) < cols; }
  // The eight values of the row (or vector) that starts at `at`; zeros past the
  // last column.
  template <bool WIDE>
  __device__ __forceinline__ void load(Raw8<WIDE>& r, const void* p, int64_t at, int kind, int c) const {
    if constexpr (VEC == 8) {
      const char* q = static_cast<const char*>(p) + (at + col(c, 0)) * (WIDE ? 4 : 2);
#pragma unroll
      for (int i = 0; i < (WIDE ? 2 : 1); ++i)
        r.q[i] = in(c, 0) ? reinterpret_cast<const u32x4*>(q)[i] : u32x4{0u, 0u, 0u, 0u};
    } else {
      static_assert(VEC == 8 || WIDE, "single columns are loaded as floats");
      // no branch between the loads, so that all of them are in flight
      uint32_t x[8];
      if (kind == kOutF32) {
        const uint32_t* q = static_cast<const uint32_t*>(p) + at;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = q[min(col(c, j), cols - 1)];
      } else {
        const uint16_t* q = static_cast<const uint16_t*>(p) + at;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = q[min(col(c, j), cols - 1)];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[j] = kind == kOutF16 ? __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)x[j])) : x[j] << 16;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) r.q[j / 4][j % 4] = in(c, j) ? x[j] : 0u;
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t at, int kind, int c, const float* x) const {
    if constexpr (VEC == 8) {
      if (in(c, 0)) store8(p, at + col(c, 0), x, kind);
    } else {
      if (kind == kOutF32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (in(c, j)) static_cast<float*>(p)[at + col(c, j)] = x[j];
        }
      } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = pack16(x[2 * k], x[2 * k + 1], kind == kOutF16);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (in(c, j)) static_cast<uint16_t*>(p)[at + col(c, j)] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
        }
      }
    }
  }
};

// Sum over the threads of a row (ONE: one wave, else the block's up to 16
// waves), in every one of them.
template <bool ONE>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (!ONE) {
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    if (lane == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (lane & 15) < waves ? red[lane & 15] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  }
  return v;
}

// BW, RW, WW: block, residual and weights are fp32.
template <int VEC, int CH, bool ONE, bool BW, bool RW, bool WW>
__global__ __launch_bounds__(ONE ? 256 : 1024) void vq_norm_kernel(NormArgs a) {
  __shared__ float red[2][16];
  // With eight values a thread (few rows in flight) the weights are loaded up
  // front too, so one memory latency covers every input.
  constexpr bool kEarly = CH == 1;
  const int tid = ONE ? threadIdx.x & 63 : threadIdx.x;
  const int64_t t = ONE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (t >= a.T) return;  // whole waves, and only where a row is one wave
  const RowMap<VEC> m{tid, ONE ? 64 : (int)blockDim.x, a.cols};
  const int64_t at = t * a.cols;
  Raw8<BW> rb[CH];
  Raw8<RW> rr[CH];
  Raw8<WW> rw, rp;
  if (a.block) {
#pragma unroll
    for (int c = 0; c < CH; ++c) m.load(rb[c], a.block, at, a.block_kind, c);
  }
  if (a.residual) {
#pragma unroll
    for (int c = 0; c < CH; ++c) m.load(rr[c], a.residual, at, a.res_kind, c);
  }
  if (kEarly && a.post_w) m.load(rw, a.post_w, 0, a.w_kind, 0);
  if (kEarly && a.pre_w) m.load(rp, a.pre_w, 0, a.w_kind, 0);
  float g1 = a.alpha;
  if (a.gate_kind == kGateToken) g1 *= gate_act(load1(a.gate, t, a.w_kind), a.gate_act);
  float v[CH][8];
  if (a.block) {
#pragma unroll
    for (int c = 0; c < CH; ++c) to_float(rb[c], a.block_kind, v[c]);
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = 0.0f;
    }
  }
  if (a.post_w) {
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(v[c][j], v[c][j], s);
    }
    g1 *= 1.0f / sqrtf(row_sum<ONE>(s, red[0]) * a.inv_cols + a.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float w[8];
      if (!kEarly) m.load(rw, a.post_w, 0, a.w_kind, c);
      to_float(rw, a.w_kind, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= w[j] + a.offset;
    }
  }
  if (a.gate_kind == kGateChannel || a.gate_kind == kGateFull) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      Raw8<WW> rg;
      float g[8];
      m.load(rg, a.gate, a.gate_kind == kGateFull ? at : 0, a.w_kind, c);
      to_float(rg, a.w_kind, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= gate_act(g[j], a.gate_act);
    }
  }
  if (a.residual) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float x[8];
      to_float(rr[c], a.res_kind, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = fmaf(a.beta, x[j], v[c][j] * g1);
    }
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= g1;
    }
  }
  if (a.v_out) {
#pragma unroll
    for (int c = 0; c < CH; ++c) m.store(a.v_out, at, a.res_kind, c, v[c]);
  }
  if (!a.h) return;
  // past the last column v is zero, but for a post norm of infinities
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s = m.in(c, j) ? fmaf(v[c][j], v[c][j], s) : s;
  }
  const float r = 1.0f / sqrtf(row_sum<ONE>(s, red[1]) * a.inv_cols + a.eps);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (a.pre_w) {
      float w[8];
      if (!kEarly) m.load(rp, a.pre_w, 0, a.w_kind, c);
      to_float(rp, a.w_kind, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= r * (w[j] + a.offset);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= r;
    }
    if (VEC == 8 && a.h_kind == kNormE4m3) {
      // 16 lanes side by side hold a block of 128 columns
      if (!m.in(c, 0)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = 0.0f;
      }
      float sc;
      const u32x2 q = fp8_quantize8(v[c], abs_max8(v[c]), &sc);
      if (m.in(c, 0)) {
        *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.h) + at + m.col(c, 0)) = q;
        if ((tid & 15) == 0) a.h_scales[t * a.kb + m.col(c, 0) / kFp8Block] = sc;
      }
    } else {
      m.store(a.h, at, a.h_kind, c, v[c]);
    }
  }
}

template <int VEC, int CH, bool ONE, bool BW, bool RW, bool WW>
void run(const NormArgs& a, hipStream_t s) {
  // whole waves for the row's pieces of 8, split over CH chunks
  const int pieces = (a.cols + 7) / 8, threads = ONE ? 256 : ((pieces + CH - 1) / CH + 63) / 64 * 64;
  const unsigned blocks = ONE ? ((unsigned)a.T + 3) / 4 : (unsigned)a.T;
  hipLaunchKernelGGL((vq_norm_kernel<VEC, CH, ONE, BW, RW, WW>), dim3(blocks), dim3(threads), 0, s, a);
}

template <int CH, bool ONE>
void run_types(const NormArgs& a, hipStream_t s) {
  const int w = (a.block && a.block_kind == kOutF32 ? 4 : 0) | (a.residual && a.res_kind == kOutF32 ? 2 : 0) |
                (a.w_kind == kOutF32 ? 1 : 0);
  switch (w) {
    case 0: return run<8, CH, ONE, false, false, false>(a, s);
    case 1: return run<8, CH, ONE, false, false, true>(a, s);
    case 2: return run<8, CH, ONE, false, true, false>(a, s);
    case 3: return run<8, CH, ONE, false, true, true>(a, s);
    case 4: return run<8, CH, ONE, true, false, false>(a, s);
    case 5: return run<8, CH, ONE, true, false, true>(a, s);
    case 6: return run<8, CH, ONE, true, true, false>(a, s);
    default: return run<8, CH, ONE, true, true, true>(a, s);
  }
}

void run_norm(const NormArgs& a, hipStream_t s) {
  const int pieces = (a.cols + 7) / 8;
  // single columns, coalesced over the threads (1 x 5119: 5.6 us, 4096 x 5119:
  // 72 to 75; with a branch on the type at every load they took 25 and 152)
  if (a.cols % 8 != 0) {
    if (pieces <= 1024) return run<1, 1, false, true, true, true>(a, s);
    if (pieces <= 2048) return run<1, 2, false, true, true, true>(a, s);
    return run<1, 4, false, true, true, true>(a, s);
  }
  if (pieces <= 64) return run_types<1, true>(a, s);
  // 8 values a thread while that many threads run at once, then 16: fewer
  // reductions a value (4096 x 5120 bf16: 41.8 against 49.6 us, 8192 x 2048:
  // 31.6 against 33.2; 512 x 5120: 10.2 against 9.7, one row of 5120: 6.2
  // against 5.0; 24 values: 42.4 at 4096 x 5120)
  const bool many = (int64_t)a.T * a.cols >= (int64_t)8 << 20;
  if (pieces <= 1024 && !many) return run_types<1, false>(a, s);
  if (pieces <= 2048) return run_types<2, false>(a, s);
  return run_types<4, false>(a, s);
}

}  // namespace

hipError_t launch_norm(const NormSpec& n, const void* block, const void* residual, int T, void* v_out, void* h,
                       float* h_scales, hipStream_t s) {
  NormArgs a{};
  a.block = block;
  a.residual = residual;
  a.post_w = n.post_w;
  a.pre_w = n.pre_w;
  a.gate = n.gate;
  a.v_out = v_out;
  a.h = h;
  a.h_scales = h_scales;
  a.T = T;
  a.cols = n.cols;
  a.kb = (n.cols + kFp8Block - 1) / kFp8Block;
  a.block_kind = n.block_kind;
  a.res_kind = n.res_kind;
  a.w_kind = n.w_kind;
  a.h_kind = n.h_kind;
  a.gate_kind = n.gate_kind;
  a.gate_act = n.gate_act;
  a.alpha = n.alpha;
  a.beta = n.beta;
  a.eps = n.eps;
  a.offset = n.offset;
  a.inv_cols = 1.0f / (float)n.cols;
  run_norm(a, s);
  return hipGetLastError();
}

}  // namespace vqmi
