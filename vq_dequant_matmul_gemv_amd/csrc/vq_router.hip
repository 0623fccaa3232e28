// vq_router.hip -- routing to experts: from a router's logits to the expert
// ids and route weights the routed products (vq_moe_gemv, vq_moe_gemm) take.
//
// The mathematics, per token with logits l_e:
//   p_e   = softmax over the experts still in play, or 1 / (1 + exp(-l_e))
//   key_e = l_e without a bias (both scores rise with l_e, so the order of the
//           logits is the order of the scores, exactly), p_e + bias_e with one
//   group score = the largest key of the group, or the sum of its two largest
//           (of p_e without a bias); the best top_groups groups stay
//   the top_k largest keys, ties to the lowest expert, in descending order
//   weight = scale * p_e, or scale * p_e / (the chosen ones' sum)
//
// One wave per token: lane i holds experts i*PL .. i*PL + PL - 1 (PL = 1 ...
// 16), so among equal keys the lowest lane, then the lowest register, is the
// lowest expert.  A choice is a maximum over the lane's keys, a maximum over
// the wave on order-preserving integer keys (DPP, no LDS), and one ballot.
#include "vq_device.h"
#include "vq_kernels.h"

#include <cfloat>

namespace vqmi {

namespace {

constexpr int kRouterWaves = 4;  // tokens per block

// Floats and doubles as unsigned integers of the same order, never 0 for a
// number above -inf: 0 stands for "out of play".  -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double f) {
  const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
  return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
// Largest value of the wave, in every lane (row shifts by 1, 2, 4, 8, then
// the two row broadcasts; lane 63 ends with the whole wave's maximum).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, dpp_u32<0x111>(v));
  v = max(v, dpp_u32<0x112>(v));
  v = max(v, dpp_u32<0x114>(v));
  v = max(v, dpp_u32<0x118>(v));
  v = max(v, dpp_u32<0x142>(v));
  v = max(v, dpp_u32<0x143>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  const uint32_t hi = wave_max((uint32_t)(v >> 32));
  const uint32_t lo = wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ float wave_maxf(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

struct RouterArgs {
  const void* logits;
  const float* bias;   // nullptr: none
  int32_t* ids;
  float* weights;
  int T, E, top_k;
  int sigmoid;         // else softmax
  int groups, top_groups, group_size, top2;
  int lanes_per_group;  // 64 / (groups rounded up to a power of two)
  int renorm, vec;     // vec: a lane's PL logits are one aligned piece
  float scale;
};

template <int DT>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
  if constexpr (DT == kOutF32) return static_cast<const float*>(p)[i];
  else if constexpr (DT == kOutF16) return (float)static_cast<const _Float16*>(p)[i];
  else return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// The score of one expert, in 64 bits (exact enough to order any two keys
// that are not equal by construction).
__device__ __forceinline__ double score64(float l, bool sigmoid, double m, double inv_z) {
  return sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - m) * inv_z;
}

template <int PL, int DT>
__global__ __launch_bounds__(64 * kRouterWaves) void vq_router_kernel(RouterArgs a) {
  __shared__ double lds[kRouterWaves][64 * PL];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kRouterWaves + wave;
  if (t >= a.T) return;  // whole waves; no block barriers below
  const int E = a.E, e0 = lane * PL;
  const int64_t row = t * E;

  float l[PL];
  bool live[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = e0 + i;
    const float v = e < E ? logit_at<DT>(a.logits, row + e) : -INFINITY;
    live[i] = v > -INFINITY;  // false for NaN too
    if (a.bias && e < E) live[i] = live[i] && a.bias[e] > -INFINITY;
    l[i] = fminf(fmaxf(v, -FLT_MAX), FLT_MAX);
  }

  const bool need_p = a.bias || (a.groups > 1 && a.top2);
  const bool sigmoid = a.sigmoid != 0;
  double p[PL];
  double m = 0.0, inv_z = 0.0;
  if (!sigmoid) {
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < PL; ++i) mx = live[i] ? fmaxf(mx, l[i]) : mx;
    mx = wave_maxf(mx);
    m = mx;
    if (need_p || !a.renorm) {
      double z = 0.0;
#pragma unroll
      for (int i = 0; i < PL; ++i) z += live[i] ? exp((double)l[i] - m) : 0.0;
      z = wave_sum(z);
      inv_z = z > 0.0 ? 1.0 / z : 0.0;
    }
  }
  uint64_t key[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    p[i] = need_p && live[i] ? score64(l[i], sigmoid, m, inv_z) : 0.0;
    const double k = a.bias ? p[i] + (double)(e0 + i < E ? a.bias[e0 + i] : 0.0f) : (double)l[i];
    key[i] = live[i] ? order_key(k) : 0ull;
  }

  if (a.groups > 1) {
    // group scores: the wave's lanes split over the groups, each lane scans
    // its share of a group's values in LDS, then its group's lanes combine
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      double v = -INFINITY;
      if (live[i]) v = a.bias ? p[i] + (double)a.bias[e0 + i] : (a.top2 ? p[i] : (double)l[i]);
      lds[wave][e0 + i] = v;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const int lpg = a.lanes_per_group, g = lane / lpg, sub = lane % lpg;
    double m1 = -INFINITY, m2 = -INFINITY;
    if (g < a.groups) {
      for (int j = sub; j < a.group_size; j += lpg) {
        const double v = lds[wave][g * a.group_size + j];
        m2 = fmax(m2, fmin(m1, v));
        m1 = fmax(m1, v);
      }
    }
    for (int o = 1; o < lpg; o <<= 1) {
      const double b1 = __shfl_xor(m1, o, 64), b2 = __shfl_xor(m2, o, 64);
      m2 = fmax(fmin(m1, b1), fmax(m2, b2));
      m1 = fmax(m1, b1);
    }
    const double s = a.top2 && m2 > -INFINITY ? m1 + m2 : m1;
    const uint64_t gk = g < a.groups && m1 > -INFINITY ? order_key(s) : 0ull;
    int rank = 0;
    for (int h = 0; h < a.groups; ++h) {
      const uint64_t o = __shfl(gk, h * lpg, 64);
      rank += (o > gk || (o == gk && h < g)) ? 1 : 0;
    }
    const uint64_t keep = __ballot(gk != 0 && rank < a.top_groups);
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = e0 + i;
      const int ge = e / a.group_size;
      if (e >= E || !(keep >> (ge * lpg) & 1)) key[i] = 0ull;
    }
  }

  int my_id = -1;
  float my_l = -INFINITY;
  for (int j = 0; j < a.top_k; ++j) {
    uint64_t best = 0ull;
    int at = 0;
    float bl = 0.0f;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      if (key[i] > best) { best = key[i]; at = i; bl = l[i]; }
    }
    const uint64_t top = wave_max(best);
    if (top == 0ull) break;
    const uint64_t who = __ballot(best == top);
    const int src = __ffsll((unsigned long long)who) - 1;
    const int id = __shfl(e0 + at, src, 64);
    const float chosen = __shfl(bl, src, 64);
    if (lane == src) {
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        if (i == at) key[i] = 0ull;
      }
    }
    if (lane == j) { my_id = id; my_l = chosen; }
  }

  if (lane < a.top_k) {
    a.ids[t * a.top_k + lane] = my_id;
  }
  double w = my_id >= 0 ? score64(my_l, sigmoid, m, a.renorm ? 1.0 : inv_z) : 0.0;
  if (a.renorm) {
    const double sum = wave_sum(w);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (lane < a.top_k) a.weights[t * a.top_k + lane] = (float)(w * a.scale);
}

template <int PL>
hipError_t run_router(const RouterArgs& a, int dtype, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + kRouterWaves - 1) / kRouterWaves)), block(64 * kRouterWaves);
  if (dtype == kOutF32) hipLaunchKernelGGL((vq_router_kernel<PL, kOutF32>), grid, block, 0, s, a);
  else if (dtype == kOutF16) hipLaunchKernelGGL((vq_router_kernel<PL, kOutF16>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((vq_router_kernel<PL, kOutBF16>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_router(const RouterSpec& r, const void* logits, int T, int32_t* ids, float* weights,
                         hipStream_t s) {
  RouterArgs a{};
  a.logits = logits;
  a.bias = r.bias;
  a.ids = ids;
  a.weights = weights;
  a.T = T;
  a.E = r.num_experts;
  a.top_k = r.top_k;
  a.sigmoid = r.sigmoid;
  a.groups = r.groups;
  a.top_groups = r.top_groups;
  a.group_size = r.num_experts / r.groups;
  a.top2 = r.top2;
  int pow2 = 1;
  while (pow2 < r.groups) pow2 <<= 1;
  a.lanes_per_group = 64 / pow2;
  a.renorm = r.renorm;
  a.scale = r.scale;
  const int pl = (r.num_experts + 63) / 64;
  if (pl <= 1) return run_router<1>(a, r.logits_kind, s);
  if (pl <= 2) return run_router<2>(a, r.logits_kind, s);
  if (pl <= 4) return run_router<4>(a, r.logits_kind, s);
  if (pl <= 8) return run_router<8>(a, r.logits_kind, s);
  return run_router<16>(a, r.logits_kind, s);
}

}  // namespace vqmi
