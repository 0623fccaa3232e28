// vq_mx4_moe.hip -- a mixture-of-experts layer for a few tokens over 4-bit
// experts: behind the routing, one kernel for the gate and up projections with
// SwiGLU and one for the down projection with the weighted sum.
//
//   h[t][s] = silu(W_gate[e] x_t) * (W_up[e] x_t),   e = ids[t][s]
//   y[t]    = sum over the slots s of weight[t][s] * W_down[e] h[t][s]
//
// Bound by the bytes of the experts that the tokens hit, so each expert's
// weights are read once: the tokens that chose it are the columns of its
// matrix products.
#include "vq_block_kernels.h"
#include "vq_mx4_device.h"
#include "vq_store_device.h"

namespace vqmi {

namespace {

struct MoeArgs {
  const uint8_t *gu, *gus, *dn, *dns;  // gate and up rows in turn, down: values and scales
  const void* x;
  void* y;
  const int32_t* ids;
  const float* weights;
  int32_t* leads;  // [pairs]: 1 where a pair is its expert's first
  uint16_t* h;     // [kMx4Planes][pairs][inter]
  int T, top_k, pairs;
  int hidden_blocks, inter_blocks;  // blocks of 32 columns
  int y_kind;
  int whole_gu, whole_dn;
};

// fp32 as three bf16 values whose sum it is: its 24 bits, 8 at a time.
// Infinities and NaN lie in the first.
__device__ __forceinline__ void split_planes(float v, uint32_t* p) {
  const uint32_t a = __float_as_uint(v) & 0xffff0000u;
  const float rest = v - __uint_as_float(a);
  const uint32_t b = __float_as_uint(rest) & 0xffff0000u;
  const float last = rest - __uint_as_float(b);
  const bool finite = fabsf(v) < INFINITY;
  p[0] = v == v ? a >> 16 : 0x7fc0u;
  p[1] = finite ? b >> 16 : 0u;
  p[2] = finite ? __float_as_uint(last) >> 16 : 0u;
}

// Gate and up: a block takes 16 rows of the expert of pair blockIdx.y, if that
// pair is the expert's first, for all pairs of the expert.
template <int XK, int WAVES, int PCS, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void vq_mx4_moe_up_kernel(MoeArgs a) {
  constexpr int kStep = 4 * PCS;
  __shared__ float4_t part[WAVES][64];
  __shared__ uint16_t members[kMx4MoePairs];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int pair = blockIdx.y, e = a.ids[pair];
  int count = 0;
  bool lead = e >= 0;
  for (int base = 0; base < a.pairs; base += 64) {
    const int q = base + lane;
    const bool mine = q < a.pairs && a.ids[q] == e;
    const uint64_t m = __ballot(mine);
    if (__ballot(mine && q < pair) != 0ull) lead = false;
    if (wave == 0 && mine) members[count + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)q;
    count += __popcll(m);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.leads[pair] = lead ? 1 : 0;
  if (!lead) return;
  __syncthreads();
  const int r = lane & 15, g = lane >> 4, r0 = blockIdx.x * 16;
  const uint32_t blocks = a.hidden_blocks;
  const int64_t row0 = (int64_t)e * a.inter_blocks * 64 + r0;  // 2 * inter rows an expert
  const rsrc_t wr = make_rsrc(a.gu + row0 * blocks * 16, (uint64_t)16 * blocks * 16);
  const rsrc_t wsr = make_rsrc(a.gus + row0 * blocks, (uint64_t)16 * blocks);
  const rsrc_t xr = make_rsrc(a.x, (uint64_t)a.T * blocks * 64);
  const uint32_t steps = (blocks + kStep - 1) / kStep;
  for (int m0 = 0; m0 < count; m0 += 16) {
    const int mine = m0 + r < count ? members[m0 + r] : -1;
    const uint32_t xrow = mine >= 0 ? (uint32_t)(mine / a.top_k) * blocks * 64u : kOutOfRange;
    Mx4Step<XK, PCS, 1> st[DEPTH];
    float4_t acc[1] = {{0.0f, 0.0f, 0.0f, 0.0f}};
    auto load = [&](int j, uint32_t k) {
      const uint32_t b = k * kStep + g * PCS;
      mx4_load(st[j].w, wr, wsr, r, b, blocks, blocks, a.whole_gu);
      mx4_load_x(st[j].x[0], xr, xrow, 0u, b, blocks);
    };
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) load(j, wave + j * WAVES);
    for (uint32_t k = wave; k < steps; k += DEPTH * WAVES) {
#pragma unroll
      for (int j = 0; j < DEPTH; ++j) {
        st[j].dot(acc);
        load(j, k + (j + DEPTH) * WAVES);
      }
    }
    if (m0 > 0) __syncthreads();  // the sums of the members before have been read
    part[wave][lane] = acc[0];
    __syncthreads();
    if (wave == 0 && mine >= 0) {
      float4_t s = part[0][lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) s += part[w][lane];
      uint32_t lo[kMx4Planes], hi[kMx4Planes];
      split_planes(silu_mul<true>(s[0], s[1]), lo);
      split_planes(silu_mul<true>(s[2], s[3]), hi);
      const int64_t inter = (int64_t)a.inter_blocks * 32;
      uint16_t* out = a.h + mine * inter + r0 / 2 + 2 * g;
#pragma unroll
      for (int p = 0; p < kMx4Planes; ++p)
        *reinterpret_cast<uint32_t*>(out + p * a.pairs * inter) = lo[p] | hi[p] << 16;
    }
  }
}

// Down: a block takes 16 output rows for all tokens, its waves the experts in
// turn.  The columns of a wave's products are the tokens themselves, 16 a tile:
// those that did not choose the expert multiply zeros and leave the sum as it
// is.
template <int WAVES, int NT, int PCS>
__global__ __launch_bounds__(64 * WAVES) void vq_mx4_moe_down_kernel(MoeArgs a) {
  constexpr int kStep = 4 * PCS;
  __shared__ float4_t part[WAVES][NT][64];
  __shared__ int32_t ids[kMx4MoePairs];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4, r0 = blockIdx.x * 16;
  for (int p = threadIdx.x; p < a.pairs; p += 64 * WAVES) ids[p] = a.ids[p];
  __syncthreads();
  const uint32_t blocks = a.inter_blocks;
  const uint32_t plane = (uint32_t)a.pairs * blocks * 64u;  // bytes
  const rsrc_t hr = make_rsrc(a.h, (uint64_t)kMx4Planes * plane);
  const uint32_t steps = (blocks + kStep - 1) / kStep;
  float4_t acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  int turn = 0;  // experts seen
  for (int base = 0; base < a.pairs; base += 64) {
    uint64_t todo = __ballot(base + lane < a.pairs && a.leads[min(base + lane, a.pairs - 1)] != 0);
    for (; todo != 0ull; todo &= todo - 1, ++turn) {
      if (turn % WAVES != wave) continue;
      const int e = __builtin_amdgcn_readfirstlane(ids[base + __builtin_ctzll(todo)]);
      int mine[NT];
      uint32_t xrow[NT];
      bool any[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int t = 16 * n + r;
        mine[n] = -1;
        for (int s = 0; s < a.top_k; ++s) {
          const int p = t * a.top_k + s;
          if (t < a.T && ids[p] == e) mine[n] = p;
        }
        xrow[n] = mine[n] >= 0 ? (uint32_t)mine[n] * blocks * 64u : kOutOfRange;
        any[n] = __ballot(mine[n] >= 0) != 0ull;
      }
      const int64_t row0 = (int64_t)e * a.hidden_blocks * 32 + r0;
      const rsrc_t wr = make_rsrc(a.dn + row0 * blocks * 16, (uint64_t)16 * blocks * 16);
      const rsrc_t wsr = make_rsrc(a.dns + row0 * blocks, (uint64_t)16 * blocks);
      float4_t d[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) d[n] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
      for (uint32_t k = 0; k < steps; ++k) {
        const uint32_t b = k * kStep + g * PCS;
        Mx4Frag<PCS> w;
        mx4_load(w, wr, wsr, r, b, blocks, blocks, a.whole_dn);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (!any[n]) continue;
          Mx4XFrag<PCS, kMx4Planes> x;
          mx4_load_x(x, hr, xrow[n], plane, b, blocks);
          mx4_dot16s<kMx4XPlanes, 1>(w, &x, &d[n], false);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (mine[n] < 0) continue;
        const float f = a.weights[mine[n]];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = fmaf(f, d[n][i], acc[n][i]);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) part[wave][n][lane] = acc[n];
  __syncthreads();
  for (int n = wave; n < NT; n += WAVES) {  // a wave joins a tile of tokens
    float4_t s = part[0][n][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += part[w][n][lane];
    const int t = 16 * n + r;
    if (t >= a.T) continue;
    const int64_t at = (int64_t)t * a.hidden_blocks * 32 + r0 + 4 * g;
    const float v[4] = {s[0], s[1], s[2], s[3]};
    store_run<4>(a.y, at, v, a.y_kind);
  }
}

constexpr size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }

}  // namespace

size_t mx4_moe_workspace_bytes(int T, int top_k, int inter) {
  const size_t pairs = (size_t)T * top_k;
  return align16(pairs * sizeof(int32_t)) + kMx4Planes * pairs * inter * sizeof(uint16_t);
}

hipError_t launch_mx4_moe(const RouterSpec& r, const Mx4View& gate_up, const Mx4View& down, const void* logits,
                          const void* x, int x_kind, int T, void* y, int y_kind, int32_t* ids, float* weights,
                          void* workspace, hipStream_t s) {
  hipError_t e = launch_router(r, logits, T, ids, weights, s);
  if (e != hipSuccess) return e;
  MoeArgs a{};
  a.gu = gate_up.values;
  a.gus = gate_up.scales;
  a.dn = down.values;
  a.dns = down.scales;
  a.x = x;
  a.y = y;
  a.ids = ids;
  a.weights = weights;
  a.T = T;
  a.top_k = r.top_k;
  a.pairs = T * r.top_k;
  a.leads = static_cast<int32_t*>(workspace);
  a.h = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + align16((size_t)a.pairs * sizeof(int32_t)));
  a.hidden_blocks = gate_up.cols / kMx4Block;
  a.inter_blocks = down.cols / kMx4Block;
  a.y_kind = y_kind;
  auto whole = [](const uint8_t* q, int blocks) { return blocks % 4 == 0 && reinterpret_cast<uintptr_t>(q) % 4 == 0; };
  a.whole_gu = whole(gate_up.scales, a.hidden_blocks);
  a.whole_dn = whole(down.scales, a.inter_blocks);
  const dim3 up((unsigned)a.inter_blocks * 4, (unsigned)a.pairs);
  if (x_kind == kMx4XF16) hipLaunchKernelGGL((vq_mx4_moe_up_kernel<kMx4XF16, 4, 2, 2>), up, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((vq_mx4_moe_up_kernel<kMx4XBF16, 4, 2, 2>), up, dim3(256), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)a.hidden_blocks * 2);
  if (T <= 16) hipLaunchKernelGGL((vq_mx4_moe_down_kernel<8, 1, 2>), grid, dim3(512), 0, s, a);
  else if (T <= 32) hipLaunchKernelGGL((vq_mx4_moe_down_kernel<8, 2, 2>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((vq_mx4_moe_down_kernel<8, 4, 2>), grid, dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace vqmi
