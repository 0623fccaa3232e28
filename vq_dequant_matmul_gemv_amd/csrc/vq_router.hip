// vq_router.hip -- routing to experts: from a router's logits to the expert
// ids and route weights the routed products (vq_moe_gemv, vq_moe_gemm) take.
// The mathematics and a wave's work stand in vq_router_device.h.
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
#include "vq_router_device.h"

namespace vqmi {

namespace {

constexpr int kRouterWaves = 4;  // per block; a wave routes 64 / LPT tokens

template <int LPT, int PL, int DT>
__global__ __launch_bounds__(64 * kRouterWaves) void vq_router_kernel(RouterArgs a) {
  __shared__ double lds[kRouterWaves][kRouteLds<LPT, PL>];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = ((int64_t)blockIdx.x * kRouterWaves + wave) * (64 / LPT);
  if (t0 < a.T) route_wave<LPT, PL, DT>(a, lds[wave], t0, threadIdx.x & 63);  // whole waves; no block barriers inside
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

RouterPlan router_plan(const RouterSpec& r, const void* logits, int T, int32_t* ids, float* weights) {
  RouterPlan p{};
  RouterArgs& a = p.args;
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
  p.lanes = lpt;
  p.per_lane = pl;
  return p;
}

hipError_t launch_router(const RouterSpec& r, const void* logits, int T, int32_t* ids, float* weights,
                         hipStream_t s) {
  const RouterPlan p = router_plan(r, logits, T, ids, weights);
  if (p.lanes == 16) return run_lanes<16>(p.args, p.per_lane, r.logits_kind, s);
  if (p.lanes == 32) return run_lanes<32>(p.args, p.per_lane, r.logits_kind, s);
  return run_lanes<64>(p.args, p.per_lane, r.logits_kind, s);
}

}  // namespace vqmi
