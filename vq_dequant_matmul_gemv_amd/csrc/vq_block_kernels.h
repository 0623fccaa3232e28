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
// Tensors of 4-bit e2m1 values with a scale for each 32 columns (vq_mx4.hip).
struct Mx4View {
  const uint8_t* values;
  const uint8_t* scales;
  int rows, cols;
};
hipError_t launch_mx4_quant(const void* x, int x_kind, int64_t values, uint8_t* q, uint8_t* scales, hipStream_t s);
hipError_t launch_mx4_dequant(const uint8_t* q, const uint8_t* scales, int64_t values, void* y, int y_kind,
                              hipStream_t s);
// What the activations of a product are (kMx4XPlanes: fp32 as three bf16 planes).
enum Mx4X { kMx4XMx4 = 0, kMx4XF16 = 1, kMx4XBF16 = 2, kMx4XPlanes = 3 };
struct Mx4Plan {
  int kernel = -1;  // -1: no kernel holds these sizes in one launch
  int splits = 1, split_blocks = 0;
  size_t workspace = 0;
};
// The plans for these sizes with 4-bit and with 16-bit activations.  A call looks
// them up once and runs what it has checked its workspace for.
struct Mx4Plans {
  Mx4Plan mx4, x16;
  size_t workspace() const { return mx4.workspace > x16.workspace ? mx4.workspace : x16.workspace; }
};
Mx4Plans mx4_plans(int rows, int cols, int T);
hipError_t launch_mx4_gemm(const Mx4View& w, const IoSpec& io, const Mx4Plan& p, const void* x, int x_kind,
                           const uint8_t* xs, int T, void* y, void* workspace, hipStream_t s);
// A mixture-of-experts layer for a few tokens (vq_mx4_moe.hip); gate_up and
// down: num_experts stacked matrices, rows and cols those of one.
constexpr int kMx4MoeTokens = 64;
constexpr int kMx4MoePairs = 1024;  // T * top_k
constexpr int kMx4MoeExperts = 1024;  // the router's limit
size_t mx4_moe_workspace_bytes(int T, int top_k, int hidden, int inter);
hipError_t launch_mx4_moe(const RouterSpec& r, const Mx4View& gate_up, const Mx4View& down, const void* logits,
                          const void* x, int x_kind, int T, void* y, int y_kind, int32_t* ids, float* weights,
                          void* workspace, hipStream_t s);

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
