// vq_norm.hip -- the norms before and after a block, fused with its gate and
// the scaled residual sum, and with the quantization of the next input.
//
//   u = block * rsqrt(mean(block^2) + eps) * (post_weight + offset)   (or block as it is)
//   v = beta * residual + alpha * act(gate) * u
//   h = v * rsqrt(mean(v^2) + eps) * (pre_weight + offset)
//
// The row stays in registers between its one read and its writes: up to 32
// values a thread, 64, 256 or 1024 threads a row.  All arithmetic and both
// sums of squares are fp32; v and h are rounded once, on their stores (h
// comes from the unrounded v).
#include "vq_fp8_device.h"
#include "vq_kernels.h"

#include <algorithm>

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

// Eight values as they lie in memory: 16 bytes, or 32 for fp32.
struct Raw8 {
  u32x4 a, b;
};

__device__ __forceinline__ Raw8 load_raw8(const void* p, int64_t i, int kind) {
  Raw8 r{};
  if (kind == kOutF32) {
    const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + i);
    r.a = q[0];
    r.b = q[1];
  } else {
    r.a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
  }
  return r;
}

__device__ __forceinline__ void raw_to_float(const Raw8& r, int kind, float* x) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  if (kind == kOutF32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  } else if (kind == kOutF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const half2_t h = __builtin_bit_cast(half2_t, w[i]);
      x[2 * i] = (float)h.x;
      x[2 * i + 1] = (float)h.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
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
  for (int k = 0; k < 4; ++k) {
    if (kind == kOutF16) w[k] = __builtin_bit_cast(uint32_t, half2_t{(_Float16)x[2 * k], (_Float16)x[2 * k + 1]});
    else w[k] = (uint32_t)f32_to_bf16_bits(x[2 * k]) | (uint32_t)f32_to_bf16_bits(x[2 * k + 1]) << 16;
  }
  *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = u32x4{w[0], w[1], w[2], w[3]};
}

__device__ __forceinline__ float gate_act(float g, int act) {
  if (act == kGateSigmoid) return 1.0f / (1.0f + expf(-g));
  if (act == kGateTanh) return tanhf(g);
  return g;
}

// VEC 8: a thread's values are runs of 8 columns, 16-byte loads (cols a
// multiple of 8).  VEC 1: any cols, one column at a time.
template <int VEC, int TPR, int CH>
struct RowMap {
  int tid, cols;
  __device__ __forceinline__ int col(int ch, int j) const {
    return VEC == 8 ? (ch * TPR + tid) * 8 + j : (ch * 8 + j) * TPR + tid;
  }
  __device__ __forceinline__ bool in(int ch, int j) const { return col(ch, VEC == 8 ? 0 : j) < cols; }
  // chunk ch's eight values of the row or vector that starts at `at`
  __device__ __forceinline__ void load(const void* p, int64_t at, int kind, int ch, float* x) const {
    if constexpr (VEC == 8) {
      Raw8 r{};
      if (in(ch, 0)) r = load_raw8(p, at + col(ch, 0), kind);
      raw_to_float(r, kind, x);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = in(ch, j) ? load1(p, at + col(ch, j), kind) : 0.0f;
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t at, int kind, int ch, const float* x) const {
    if constexpr (VEC == 8) {
      if (in(ch, 0)) store8(p, at + col(ch, 0), x, kind);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (in(ch, j)) store_out(p, at + col(ch, j), x[j], kind);
      }
    }
  }
};

// Sum over the TPR threads of a row, in every one of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) v += red[w];
  }
  return v;
}

template <int VEC, int TPR, int CH>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void vq_norm_kernel(NormArgs a) {
  __shared__ float red[2][16];
  constexpr int kRows = TPR == 64 ? 4 : 1;  // rows per block
  const int tid = threadIdx.x % TPR;
  const int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  if (t >= a.T) return;  // whole waves, and only where a row is one wave
  const RowMap<VEC, TPR, CH> m{tid, a.cols};
  const int64_t at = t * a.cols;
  float v[CH][8];
  if (a.block) {
#pragma unroll
    for (int c = 0; c < CH; ++c) m.load(a.block, at, a.block_kind, c, v[c]);
    if (a.post_w) {
      float s = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(v[c][j], v[c][j], s);
      }
      const float r = 1.0f / sqrtf(row_sum<TPR>(s, red[0]) * a.inv_cols + a.eps);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float w[8];
        m.load(a.post_w, 0, a.w_kind, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] *= r * (w[j] + a.offset);
      }
    }
    float g1 = a.alpha;
    if (a.gate_kind == kGateToken) g1 *= gate_act(load1(a.gate, t, a.w_kind), a.gate_act);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = 1.0f;
      if (a.gate_kind == kGateChannel || a.gate_kind == kGateFull) {
        m.load(a.gate, a.gate_kind == kGateFull ? at : 0, a.w_kind, c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = gate_act(g[j], a.gate_act);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= g1 * g[j];
    }
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = 0.0f;
    }
  }
  if (a.residual) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float x[8];
      m.load(a.residual, at, a.res_kind, c, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = fmaf(a.beta, x[j], v[c][j]);
    }
  }
  if (a.v_out) {
#pragma unroll
    for (int c = 0; c < CH; ++c) m.store(a.v_out, at, a.res_kind, c, v[c]);
  }
  if (!a.h) return;
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (m.in(c, j)) s = fmaf(v[c][j], v[c][j], s);
    }
  }
  const float r = 1.0f / sqrtf(row_sum<TPR>(s, red[1]) * a.inv_cols + a.eps);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.0f;
    if (a.pre_w) {
      m.load(a.pre_w, 0, a.w_kind, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] += a.offset;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[c][j] *= r * w[j];
    if (VEC == 8 && a.h_kind == kNormE4m3) {
      // 16 lanes side by side hold a block of 128 columns
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, m.in(c, 0) ? finite_abs(v[c][j]) : 0.0f);
      amax = row16_max(amax);
      const float sc = fp8_scale(amax);
      if (m.in(c, 0)) {
        *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.h) + at + m.col(c, 0)) = fp8_pack8(v[c], sc, fp8_lift(amax));
        if ((tid & 15) == 0) a.h_scales[t * a.kb + m.col(c, 0) / kFp8Block] = sc;
      }
    } else {
      m.store(a.h, at, a.h_kind, c, v[c]);
    }
  }
}

template <int VEC, int TPR>
hipError_t run_ch(const NormArgs& a, hipStream_t s) {
  constexpr int kRows = TPR == 64 ? 4 : 1;
  const dim3 grid((unsigned)((a.T + kRows - 1) / kRows)), block(TPR == 64 ? 256 : TPR);
  const int ch = (a.cols + TPR * 8 - 1) / (TPR * 8);
  if (ch <= 1) hipLaunchKernelGGL((vq_norm_kernel<VEC, TPR, 1>), grid, block, 0, s, a);
  else if (ch <= 2) hipLaunchKernelGGL((vq_norm_kernel<VEC, TPR, 2>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((vq_norm_kernel<VEC, TPR, 4>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <int VEC>
hipError_t run_norm(const NormArgs& a, hipStream_t s) {
  // one wave a row for short rows, up to 32 values a thread for the others
  if (a.cols <= 64 * 8) return run_ch<VEC, 64>(a, s);
  if (a.cols <= 256 * 32) return run_ch<VEC, 256>(a, s);
  return run_ch<VEC, 1024>(a, s);
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
  return n.cols % 8 == 0 ? run_norm<8>(a, s) : run_norm<1>(a, s);
}

}  // namespace vqmi
