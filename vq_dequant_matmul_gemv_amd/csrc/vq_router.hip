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
// LPT lanes (16, 32 or 64) per token, so a wave routes 4, 2 or 1: lane i of a
// token holds experts i*PL .. i*PL + PL - 1, so among equal keys the lowest
// lane, then the lowest register, is the lowest expert.  A choice is a maximum
// over the lane's keys and over the token's lanes (DPP rotations in rows of 16
// and lane swaps between rows: no LDS, no scalar code), then the same for the
// lowest expert that holds it.
//
// Which keys are larger has to be right, not nearly right: logits are compared
// as they are; scores (with a bias, or summed over a group's best two) are
// formed in fp32 first, whose error is bounded.  Where two that the choice
// depends on lie closer than twice that bound (about 1 token in 1000 on random
// sigmoid scores with 256 experts), 64 bits decide: among the chosen and the
// next one where that is all that is open, else over the whole token again.
// (Scores in 64 bits throughout take 37 us where this takes 19.)
//
// 16384 tokens x 256 experts: 10.6 us (softmax, top 8, bf16; 11.8 in fp32), 18
// to 20 us (sigmoid with a bias, 4 of 8 groups by their two best, top 8, fp32);
// one token 4.7 us.  The bytes
// would take 3.5: it is bound by the vector instructions of the choices, about
// 60 for each of the top_k + 1.  Few lanes with several experts each share a
// choice's lane exchanges among the wave's tokens: 33 us with a token a wave,
// 24 with two, 19 with four and the close ones put in order by one exponential
// a lane (5 us less than a token's full 64-bit pass, which the last wave of a
// launch used to end with: 2048 grouped tokens 10 to 12 -> 7.8).
#include "vq_block_device.h"
#include "vq_block_kernels.h"

#include <cfloat>

namespace vqmi {

namespace {

constexpr int kRouterWaves = 4;  // per block; a wave routes 64 / LPT tokens

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

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v)));
}

// op over LPT neighbouring lanes, in every one of them: rotations by 1, 2, 4
// and 8 within rows of 16 lanes, then swaps of rows and of halves.
template <int LPT, typename Op>
__device__ __forceinline__ uint32_t lanes_reduce(uint32_t v, Op op) {
  v = op(v, dpp_u32<0x121>(v));
  v = op(v, dpp_u32<0x122>(v));
  v = op(v, dpp_u32<0x124>(v));
  v = op(v, dpp_u32<0x128>(v));
  if constexpr (LPT >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(r[0], r[1]);
  }
  if constexpr (LPT >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = op(r[0], r[1]);
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  return lanes_reduce<LPT>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int LPT>
__device__ __forceinline__ uint32_t lanes_min(uint32_t v) {
  return lanes_reduce<LPT>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}
template <int LPT>
__device__ __forceinline__ float lanes_sum(float v) {
  return __uint_as_float(lanes_reduce<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  const uint32_t hi = lanes_max<64>((uint32_t)(v >> 32));
  const uint32_t lo = lanes_max<64>((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

struct RouterArgs {
  const void* logits;
  const float* bias;   // nullptr: none
  int32_t* ids;
  float* weights;
  int T, E, top_k;
  int sigmoid;         // else softmax
  int groups, top_groups, group_size, top2;
  int groups_pow2;     // groups rounded up to a power of two
  int renorm;
  int vec, vec_bias;   // a lane's PL logits (bias values) are one aligned piece
  float scale;
};

template <int DT>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
  if constexpr (DT == kOutF32) return static_cast<const float*>(p)[i];
  else if constexpr (DT == kOutF16) return (float)static_cast<const _Float16*>(p)[i];
  else return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// A lane's PL values of a row that starts at element `row` (-inf past the last
// expert).  vec: they are one aligned piece.
template <int PL, int DT>
__device__ __forceinline__ void load_row(const void* base, int E, bool vec, int64_t row, int e0, float* l) {
  constexpr int kBytes = PL * (DT == kOutF32 ? 4 : 2);
  if (vec) {
    uint32_t w[kBytes >= 4 ? kBytes / 4 : 1];
    {
      const char* p = static_cast<const char*>(base) + (row + min(e0, E - PL)) * (DT == kOutF32 ? 4 : 2);
      if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
          const u32x4 v = reinterpret_cast<const u32x4*>(p)[i];
          w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
      } else if constexpr (kBytes == 8) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(p);
        w[0] = v.x, w[1] = v.y;
      } else if constexpr (kBytes == 4) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      } else {
        w[0] = *reinterpret_cast<const uint16_t*>(p);
      }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      float v;
      if constexpr (DT == kOutF32) v = __uint_as_float(w[i]);
      else {
        const uint32_t h = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu;
        v = DT == kOutF16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)h) : __uint_as_float(h << 16);
      }
      l[i] = e0 < E ? v : -INFINITY;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const float v = logit_at<DT>(base, row + min(e0 + i, E - 1));
    l[i] = e0 + i < E ? v : -INFINITY;
  }
}

// An expert's logit: -inf for one out of play (a NaN or -inf logit or bias).
__device__ __forceinline__ float in_play(float l, float bias) {
  return l > -INFINITY && bias > -INFINITY ? fminf(fmaxf(l, -FLT_MAX), FLT_MAX) : -INFINITY;
}

// Slot `lane` of a token's LPT lanes: stores the chosen expert (-1: none) and
// its weight, in fp32.  Renormalised weights come from the chosen logits alone,
// relative to the largest of them, so they hold where the scores underflow
// fp32.  Zero where the score would be zero in 64 bits: a sigmoid whose exp(-l)
// overflows (l < -709.78, a score of 5.6e-309), a softmax whose exp(l - m) is
// below the smallest 64-bit number.  m, inv_z: largest logit in play and
// inverse sum of the softmax.
template <int LPT>
__device__ __forceinline__ void store_slot(const RouterArgs& a, int64_t t, int lane, int id, float l, float m,
                                           float inv_z, bool write) {
  float w = 0.0f;
  const float top = order_value(lanes_max<LPT>(id >= 0 ? order_key(l) : 0u));
  if (id >= 0) {
    if (a.sigmoid) {
      const float c = a.renorm ? fminf(top, 0.0f) : 0.0f;
      w = (l <= 0.0f ? expf(l - c) : 1.0f) / (1.0f + expf(-fabsf(l)));
      if (l < -709.78f) w = 0.0f;
    } else {
      w = a.renorm ? expf(l - top) : expf(l - m) * inv_z;
      if (l - m < -745.0f) w = 0.0f;
    }
  }
  if (a.renorm) {
    const float sum = lanes_sum<LPT>(w);
    w = sum > 0.0f ? w / sum : 0.0f;
  }
  if (write && lane < a.top_k) {
    a.ids[t * a.top_k + lane] = id;
    a.weights[t * a.top_k + lane] = w * a.scale;
  }
}

// One token by a whole wave with keys in 64 bits; lane i holds experts i, i +
// 64, ... (PS of them).  Uncommon, but one of the last waves of a launch may
// take it, so it is laid out for latency: one round of loads, then registers
// (with loops over LDS instead it took 4 us longer).
template <int PS, int DT>
__device__ __forceinline__ void route_token64(const RouterArgs& a, double* vals, int64_t t, int lane) {
  const bool sigmoid = a.sigmoid != 0;
  float l[PS], b[PS];
#pragma unroll
  for (int i = 0; i < PS; ++i) {
    const int e = min(lane + 64 * i, a.E - 1);
    l[i] = logit_at<DT>(a.logits, t * a.E + e);
    b[i] = a.bias ? a.bias[e] : 0.0f;
  }
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < PS; ++i) {
    l[i] = lane + 64 * i < a.E ? in_play(l[i], b[i]) : -INFINITY;
    mx = fmaxf(mx, l[i]);
  }
  const float m = order_value(lanes_max<64>(order_key(mx)));
  double inv_z = 0.0, p[PS];
#pragma unroll
  for (int i = 0; i < PS; ++i) {
    const double x = exp(sigmoid ? -(double)l[i] : (double)l[i] - m);
    p[i] = !(l[i] > -INFINITY) ? 0.0 : sigmoid ? 1.0 / (1.0 + x) : x;
    inv_z += p[i];
  }
  inv_z = sigmoid ? 1.0 : 1.0 / wave_sum(inv_z);  // unused where nothing is in play
#pragma unroll
  for (int i = 0; i < PS; ++i) p[i] = p[i] * inv_z + (double)b[i];
  uint64_t keep = ~0ull;
  const int lpg = 64 / a.groups_pow2;
  if (a.groups > 1) {
#pragma unroll
    for (int i = 0; i < PS; ++i)
      vals[lane + 64 * i] = !(l[i] > -INFINITY) ? -INFINITY : a.bias || a.top2 ? p[i] : (double)l[i];
    wave_lds_fence();
    const int g = lane / lpg;
    double m1 = -INFINITY, m2 = -INFINITY;
    if (g < a.groups) {
      for (int j = lane % lpg; j < a.group_size; j += lpg) {
        const double v = vals[g * a.group_size + j];
        m2 = fmax(m2, fmin(m1, v));
        m1 = fmax(m1, v);
      }
    }
    wave_lds_fence();
    for (int o = 1; o < lpg; o <<= 1) {
      const double b1 = __shfl_xor(m1, o, 64), b2 = __shfl_xor(m2, o, 64);
      m2 = fmax(fmin(m1, b1), fmax(m2, b2));
      m1 = fmax(m1, b1);
    }
    const double s = a.top2 && m2 > -INFINITY ? m1 + m2 : m1;  // -inf past the last group
    int rank = 0;
    for (int h = 0; h < a.groups; ++h) {
      const double so = __shfl(s, h * lpg, 64);
      rank += (h < g ? so >= s : so > s) ? 1 : 0;
    }
    keep = __ballot(s > -INFINITY && rank < a.top_groups);
  }
  uint64_t key[PS];
#pragma unroll
  for (int i = 0; i < PS; ++i) {
    const int e = lane + 64 * i;
    const bool in = l[i] > -INFINITY && (a.groups == 1 || (keep >> (e / a.group_size * lpg) & 1));
    key[i] = in ? order_key(a.bias ? p[i] : (double)l[i]) : 0ull;
  }
  int my_id = -1;
  for (int j = 0; j < a.top_k; ++j) {
    uint64_t best = 0ull;
    uint32_t at = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < PS; ++i) {
      if (key[i] > best) best = key[i], at = lane + 64 * i;
    }
    const uint64_t top = wave_max(best);
    if (top == 0ull) break;
    const uint32_t id = lanes_min<64>(best == top ? at : 0xffffffffu);
#pragma unroll
    for (int i = 0; i < PS; ++i) key[i] = (uint32_t)(lane + 64 * i) == id ? 0ull : key[i];
    if (lane == j) my_id = (int)id;
  }
  const float my_l = my_id >= 0 ? in_play(logit_at<DT>(a.logits, t * a.E + my_id), 0.0f) : -INFINITY;
  store_slot<64>(a, t, lane, my_id, my_l, m, (float)inv_z, true);
}

// Values o lanes apart (o a power of two) where the lanes below that distance
// hold equal values.
__device__ __forceinline__ float pair_up(float v, int o) {
  return o == 1 ? dpp_f32<0xb1>(v)       // quad_perm 1 0 3 2
         : o == 2 ? dpp_f32<0x4e>(v)     // quad_perm 2 3 0 1
         : o == 4 ? dpp_f32<0x141>(v)    // row_half_mirror
         : o == 8 ? dpp_f32<0x140>(v)    // row_mirror
                  : __shfl_xor(v, o, 64);
}

template <int LPT, int PL, int DT>
__global__ __launch_bounds__(64 * kRouterWaves) void vq_router_kernel(RouterArgs a) {
  // a token's scores in 64 bits, or the wave's tokens' in 32
  __shared__ double lds[kRouterWaves][PL * (LPT > 32 ? LPT : 32) > 64 ? PL * (LPT > 32 ? LPT : 32) : 64];
  constexpr int kTokens = 64 / LPT;  // of a wave
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane64 = threadIdx.x & 63;
  const int lane = lane64 % LPT, first = lane64 - lane;
  const int64_t t0 = ((int64_t)blockIdx.x * kRouterWaves + wave) * kTokens;
  if (t0 >= a.T) return;  // whole waves; no block barriers below
  const int64_t t_mine = t0 + lane64 / LPT, t = min(t_mine, (int64_t)a.T - 1);  // lanes past the end repeat the last
  const int E = a.E, e0 = lane * PL;

  float l[PL], b[PL];
  load_row<PL, DT>(a.logits, E, a.vec, t * E, e0, l);
#pragma unroll
  for (int i = 0; i < PL; ++i) b[i] = 0.0f;
  if (a.bias) load_row<PL, kOutF32>(a.bias, E, a.vec_bias, 0, e0, b);
#pragma unroll
  for (int i = 0; i < PL; ++i) l[i] = in_play(l[i], b[i]);

  const bool sigmoid = a.sigmoid != 0;
  const bool need_p = a.bias || (a.groups > 1 && a.top2);
  float m = -INFINITY, inv_z = 0.0f;
  if (!sigmoid) {
#pragma unroll
    for (int i = 0; i < PL; ++i) m = fmaxf(m, l[i]);
    m = order_value(lanes_max<LPT>(order_key(m)));
    if (need_p || !a.renorm) {
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const float e = __builtin_amdgcn_exp2f((l[i] - m) * 1.44269504f);  // NaN where nothing is in play
        z += l[i] > -INFINITY ? e : 0.0f;
      }
      z = lanes_sum<LPT>(z);
      inv_z = z > 0.0f ? 1.0f / z : 0.0f;
    }
  }
  // Keys in fp32.  A sigmoid is off by less than 2^-22: s (1 - s) times the
  // exponential's relative error of 1.22 |l| 2^-24 (argument) and 2^-23 makes
  // 0.77 * 2^-24, the sum below the reciprocal 2^-24, the reciprocal 2^-23.
  // The softmax's x = m - l rounds before that product: 2.22 |x| 2^-24 in the
  // argument.  Its sum Z = sum e^-x is off by less than 40 * 2^-24 of itself:
  // 2.22 * 2^-24 times the mean of x (at most the entropy's log 1024 = 6.94:
  // 15.4), 2 * 2^-24 of an exponential and 22 additions.  So a score is off by
  // less than 46 * 2^-24 of the largest possible one, 1 / Z: Z's 40, the
  // reciprocal's and the product's 2, and its own exponential's 2.22 x e^-x <=
  // 0.82 and 2.  The slack allows 64 * 2^-24 = 2^-18.  The sum with a bias adds
  // 2^-24 of itself, so two keys near v are certainly in order when they differ
  // by more than margin(v).
  const float slack = sigmoid ? 0x1p-21f : inv_z * 0x1p-17f;  // twice a score's error
  auto margin = [&](float v) { return fmaf(fabsf(v), 0x1.2p-23f, slack); };
  bool close = false;  // the whole token again in 64 bits
  float p[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) p[i] = l[i];
  if (need_p && sigmoid) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[i] * -1.44269504f));
      p[i] = l[i] > -INFINITY ? s + b[i] : -INFINITY;
    }
  } else if (need_p) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const float s = __builtin_amdgcn_exp2f((l[i] - m) * 1.44269504f) * inv_z;
      p[i] = l[i] > -INFINITY ? s + b[i] : -INFINITY;
    }
  }
  uint64_t keep = ~0ull;
  bool stays = true;
  const int lpg = LPT / a.groups_pow2;  // lanes that share a group's score
  const bool whole = a.group_size == lpg * PL;  // a group is whole lanes
  if (a.groups > 1) {
    const int g = lane / lpg;
    float m1 = -INFINITY, m2 = -INFINITY;
    auto add = [&](float v) {
      m2 = fmaxf(m2, fminf(m1, v));
      m1 = fmaxf(m1, v);
    };
    if (whole) {
#pragma unroll
      for (int i = 0; i < PL; ++i) add(p[i]);
    } else {
      float* vals = reinterpret_cast<float*>(lds[wave]) + first * PL;
#pragma unroll
      for (int i = 0; i < PL; ++i) vals[e0 + i] = p[i];
      wave_lds_fence();
      if (g < a.groups) {
        for (int j = lane % lpg; j < a.group_size; j += lpg) add(vals[g * a.group_size + j]);
      }
      wave_lds_fence();
    }
#pragma unroll
    for (int o = 1; o < LPT; o <<= 1) {
      if (o < lpg) {
        const float b1 = pair_up(m1, o), b2 = pair_up(m2, o);
        m2 = fmaxf(fminf(m1, b1), fmaxf(m2, b2));
        m1 = fmaxf(m1, b1);
      }
    }
    const float s = g < a.groups ? (a.top2 && m2 > -INFINITY ? m1 + m2 : m1) : -INFINITY;
    int rank = 0;
    auto against = [&](int h) {  // group h of every token of the wave
      uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(s), h * lpg);
#pragma unroll
      for (int k = 1; k < kTokens; ++k) {
        const uint32_t ok = (uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(s), k * LPT + h * lpg);
        o = first == k * LPT ? ok : o;
      }
      const float so = __uint_as_float(o);
      rank += (h < g ? so >= s : so > s) ? 1 : 0;
    };
    if (a.groups_pow2 >= 8) {
      for (int h = 0; h < a.groups_pow2; h += 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) against(h + i);
      }
    } else {
      for (int h = 0; h < a.groups; ++h) against(h);
    }
    stays = s > -INFINITY && rank < a.top_groups;
    if (need_p) {
      // the worst group that stays against the best that does not; a group's
      // sum is off by its two keys' errors (they may cancel) and its own, and
      // sums that may leave fp32 (a group is then not even known to be in play)
      // are left to the 64-bit pass
      const float in = order_value(lanes_min<LPT>(stays ? order_key(s) : order_key(INFINITY)));
      const float out = order_value(lanes_max<LPT>(stays ? order_key(-INFINITY) : order_key(s)));
      if (a.top2) {
        const float both = m1 > -INFINITY ? fabsf(m1) + (m2 > -INFINITY ? fabsf(m2) : 0.0f) : 0.0f;
        const float mag = __uint_as_float(lanes_max<LPT>(__float_as_uint(both)));
        close = in - out <= fmaf(mag, 0x1.2p-22f, 2.0f * slack) || !(mag < 0x1p126f);
      } else {
        close = in < INFINITY && in - out <= margin(in);
      }
    }
    keep = __ballot(stays) >> first;
  }
  uint32_t key[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const float v = a.bias ? p[i] : l[i];
    key[i] = l[i] > -INFINITY ? order_key(v) : 0u;
  }
  if (a.groups > 1 && whole) {
#pragma unroll
    for (int i = 0; i < PL; ++i) key[i] = stays ? key[i] : 0u;
  } else if (a.groups > 1) {
    int ge = e0 / a.group_size, left = (ge + 1) * a.group_size - e0;  // e0's group, experts left in it
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      key[i] = (keep >> (ge * lpg & 63)) & 1 ? key[i] : 0u;
      --left;
      ge += left == 0 ? 1 : 0;
      left = left == 0 ? a.group_size : left;
    }
  }
  int my_id = -1;  // with a bias also the best one left out, in lane top_k
  float last = INFINITY, last2 = INFINITY;
  bool mixed = false;  // two neighbours among them are close
  const int rounds = a.bias ? a.top_k + 1 : a.top_k;
  for (int j = 0; j < rounds; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < PL; ++i) best = max(best, key[i]);
    const uint32_t top = lanes_max<LPT>(best);
    uint32_t id = 0xffffffffu;
#pragma unroll
    for (int i = PL - 1; i >= 0; --i) id = key[i] == top ? (uint32_t)(e0 + i) : id;
    id = lanes_min<LPT>(id);
#pragma unroll
    for (int i = 0; i < PL; ++i) key[i] = (uint32_t)(e0 + i) == id ? 0u : key[i];
    if (a.bias && top != 0u) {
      const float v = order_value(top);
      mixed = mixed || last - v <= margin(v);
      last2 = last;
      last = v;
    }
    if (lane == j && top != 0u) my_id = (int)id;
  }
  // Where the last one in is clear of the second one left out, the chosen are
  // among those found: 64 bits put them in order, one a lane.
  const bool sort = a.bias && sigmoid && a.top_k < LPT;
  if (!sort) close = close || mixed;
  if (__builtin_expect(__ballot(mixed && !close) != 0ull, 0)) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < PL; ++i) best = max(best, key[i]);
    const uint32_t top = lanes_max<LPT>(best);
    const float v = order_value(top);
    close = close || (mixed && top != 0u && last2 - v <= margin(v));
    const float lc = my_id >= 0 ? logit_at<DT>(a.logits, t * E + my_id) : 0.0f;
    const double pc = my_id >= 0 ? 1.0 / (1.0 + exp(-(double)in_play(lc, 0.0f))) + (double)a.bias[my_id] : -INFINITY;
    int rank = 0;
    for (int j = 0; j <= a.top_k; ++j) {
      const double po = __shfl(pc, first + j, 64);
      const int io = __shfl(my_id, first + j, 64);
      rank += io >= 0 && (po > pc || (po == pc && io < my_id)) ? 1 : 0;
    }
    int* order = reinterpret_cast<int*>(lds[wave]) + first;
    order[lane] = -1;
    wave_lds_fence();
    if (my_id >= 0) order[rank] = my_id;  // rank <= top_k < LPT
    wave_lds_fence();
    if (mixed) my_id = order[lane];
    wave_lds_fence();
  }
  if (lane >= a.top_k) my_id = -1;
  constexpr uint64_t kTokenLanes = LPT == 64 ? ~0ull : (1ull << (LPT & 63)) - 1;
  const uint64_t again = __ballot(close);
  const float my_l = my_id >= 0 ? in_play(logit_at<DT>(a.logits, t * E + my_id), 0.0f) : -INFINITY;
  store_slot<LPT>(a, t, lane, my_id, my_l, m, inv_z, t_mine < a.T && (again >> first & kTokenLanes) == 0);
  if (__builtin_expect(again != 0ull, 0)) {
#pragma unroll 1
    for (int k = 0; k < kTokens; ++k) {
      if ((again >> (k * LPT) & kTokenLanes) != 0 && t0 + k < a.T)
        route_token64<(LPT * PL + 63) / 64, DT>(a, lds[wave], t0 + k, lane64);
    }
  }
}

template <int LPT, int PL>
hipError_t run_router(const RouterArgs& a, int dtype, hipStream_t s) {
  constexpr int kTokens = kRouterWaves * 64 / LPT;
  const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens)), block(64 * kRouterWaves);
  if (dtype == kOutF32) hipLaunchKernelGGL((vq_router_kernel<LPT, PL, kOutF32>), grid, block, 0, s, a);
  else if (dtype == kOutF16) hipLaunchKernelGGL((vq_router_kernel<LPT, PL, kOutF16>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((vq_router_kernel<LPT, PL, kOutBF16>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <int LPT>
hipError_t run_lanes(const RouterArgs& a, int pl, int dtype, hipStream_t s) {
  if (pl <= 1) return run_router<LPT, 1>(a, dtype, s);
  if (pl <= 2) return run_router<LPT, 2>(a, dtype, s);
  if (pl <= 4) return run_router<LPT, 4>(a, dtype, s);
  if (pl <= 8 || LPT == 32) return run_router<LPT, 8>(a, dtype, s);
  return run_router<LPT == 32 ? 64 : LPT, 16>(a, dtype, s);
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
  a.groups_pow2 = 1;
  while (a.groups_pow2 < r.groups) a.groups_pow2 <<= 1;
  a.renorm = r.renorm;
  a.scale = r.scale;
  // Lanes of a token: up to 8 experts a lane (16 above 512 experts), a lane at
  // least for every group and every slot (and the first one left out).  From
  // 8192 tokens on, where four a wave still fill the card, 129 to 256 experts
  // take 16 lanes of 16 (us, 32 lanes of 8 -> 16 of 16): softmax 12.0 -> 10.1
  // at 16384 tokens, 7.3 -> 6.6 at 8192, 5.6 -> 5.8 at 4096, 4.4 -> 5.3 at one;
  // grouped sigmoid 23.6 -> 21.8, 15.7 -> 15.8, 12.8 -> 12.3 and 6.2 -> 7.7.
  const int slots = r.top_k + (r.bias ? 1 : 0);
  int lpt = 16;
  while (lpt < 64 && (lpt * (lpt == 16 && T >= 8192 ? 16 : 8) < r.num_experts || lpt < r.groups || lpt < slots))
    lpt <<= 1;
  int pl = 1;
  while (pl * lpt < r.num_experts) pl <<= 1;
  const int piece = pl * (r.logits_kind == kOutF32 ? 4 : 2), align = piece < 16 ? piece : 16;
  a.vec = r.num_experts % pl == 0 && reinterpret_cast<uintptr_t>(logits) % align == 0;
  a.vec_bias = r.num_experts % pl == 0 && reinterpret_cast<uintptr_t>(r.bias) % (pl < 4 ? 4 * pl : 16) == 0;
  if (lpt == 16) return run_lanes<16>(a, pl, r.logits_kind, s);
  if (lpt == 32) return run_lanes<32>(a, pl, r.logits_kind, s);
  return run_lanes<64>(a, pl, r.logits_kind, s);
}

}  // namespace vqmi
