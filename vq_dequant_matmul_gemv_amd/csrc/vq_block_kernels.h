// vq_block_kernels.h -- host-side launch interface of the operators around the
// VQ products (routing, e4m3 tensors, norms), in the manner of vq_kernels.h.
#pragma once

#include "vq_kernels.h"

namespace vqmi {

// Routing from logits to expert ids and weights (vq_router.hip).
struct RouterSpec {
  int num_experts, top_k, sigmoid, logits_kind;  // logits_kind: OutKind
  int groups, top_groups, top2, renorm;
  float scale;
  const float* bias;
};
hipError_t launch_router(const RouterSpec& r, const void* logits, int T, int32_t* ids, float* weights,
                         hipStream_t s);

// e4m3 tensors with a scale for each block of 128 (vq_fp8.hip).
struct Fp8View {
  const uint8_t* values;
  const float* scales;
  int rows, cols;
};
hipError_t launch_fp8_quant(const void* x, int x_bf16, int T, int cols, uint8_t* q, float* scales, hipStream_t s);
// How a product runs: a kernel of vq_fp8.hip's table and the columns' splits.
struct Fp8Plan {
  int kernel = -1;  // -1: no kernel holds these sizes in one launch
  int splits = 1, split_steps = 0;
  size_t workspace = 0;
};
// The plans of vq_fp8_gemm and vq_fp8_gemm_fast for these sizes.  A call looks
// them up once and runs what it has checked its workspace for.
struct Fp8Plans {
  Fp8Plan exact, fast;
  size_t workspace() const { return exact.workspace > fast.workspace ? exact.workspace : fast.workspace; }
};
Fp8Plans fp8_plans(int rows, int cols, int T);
hipError_t launch_fp8_gemm(const Fp8View& w, const IoSpec& io, const Fp8Plan& p, const uint8_t* x, const float* xs,
                           int T, void* y, void* workspace, hipStream_t s);

// Norms before and after a block with its gate and residual (vq_norm.hip).
enum GateKind { kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateFull = 3 };
enum GateAct { kGateLinear = 0, kGateSigmoid = 1, kGateTanh = 2 };
constexpr int kNormE4m3 = 3;        // h_kind besides the OutKinds
constexpr int kNormMaxCols = 32768;  // a row stays in registers
struct NormSpec {
  int cols, block_kind, res_kind, w_kind, h_kind, gate_kind, gate_act;
  float alpha, beta, eps, offset;
  const void* post_w;
  const void* pre_w;
  const void* gate;
};
hipError_t launch_norm(const NormSpec& n, const void* block, const void* residual, int T, void* v_out, void* h,
                       float* h_scales, hipStream_t s);

}  // namespace vqmi
