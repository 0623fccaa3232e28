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
// pair is the expert's first, for all pairs of the expert, kRows at a time; its
// waves split the columns and join their sums in LDS.
template <int XK, int WAVES, int NL, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void vq_mx4_moe_up_kernel(MoeArgs a) {
  typedef Mx4Stream<XK, 1, NL, DEPTH> Stream;
  constexpr int kRows = Stream::Slot::kRows;
  __shared__ typename Stream::Slot slots[WAVES];
  __shared__ uint16_t members[kMx4MoePairs];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int pair = blockIdx.y, e = __builtin_amdgcn_readfirstlane(a.ids[pair]);
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
  Stream st;
  st.slot = slots + wave;
  st.first = 0;
  st.end = blocks;
  st.wr = make_rsrc(a.gu + row0 * blocks * 16, (uint64_t)16 * blocks * 16);
  st.xr = make_rsrc(a.x, (uint64_t)a.T * blocks * 64);
  st.plane = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) st.woff[i] = mx4_w_row(i, lane) * blocks * 16;
  const Mx4Scales ws(a.gus + row0 * blocks, 16 * blocks);
  st.wsr = ws.rsrc;
  st.wsoff = ws.word(mx4_s_row(lane) * blocks, lane);
  st.ws_skew = ws.skew(r * blocks);
  st.column = r & (kRows - 1);
  for (int m0 = 0; m0 < count; m0 += kRows) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int row = m0 + mx4_x_row<XK>(i, lane);
      st.xoff[i] = row < count ? (uint32_t)(members[row] / a.top_k) * blocks * 64u : kOutOfRange;
    }
    float4_t acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    st.run(acc, wave, WAVES, lane);
    __syncthreads();  // the slots are free: the waves' sums go there
    float4_t* part = reinterpret_cast<float4_t*>(slots);
    part[wave * 64 + lane] = acc[0] + acc[1];
    __syncthreads();
    if (wave == 0 && r < kRows && m0 + r < count) {
      float4_t s = part[lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) s += part[w * 64 + lane];
      uint32_t lo[kMx4Planes], hi[kMx4Planes];
      split_planes(silu_mul<true>(s[0], s[1]), lo);
      split_planes(silu_mul<true>(s[2], s[3]), hi);
      const int64_t inter = (int64_t)a.inter_blocks * 32;
      uint16_t* out = a.h + members[m0 + r] * inter + r0 / 2 + 2 * g;
#pragma unroll
      for (int p = 0; p < kMx4Planes; ++p)
        *reinterpret_cast<uint32_t*>(out + p * a.pairs * inter) = lo[p] | hi[p] << 16;
    }
    if (m0 + kRows < count) __syncthreads();
  }
}

// Down: a block takes 16 output rows for all tokens, its waves the experts in
// turn, for the pairs of an expert, kRows at a time.  A wave adds up its
// experts' weighted products per token in LDS, in the order of the pairs; the
// waves' sums are joined in their order.
template <int WAVES, int NL, int DEPTH, int TOKENS>
__global__ __launch_bounds__(64 * WAVES) void vq_mx4_moe_down_kernel(MoeArgs a) {
  typedef Mx4Stream<kMx4XPlanes, kMx4Planes, NL, DEPTH> Stream;
  constexpr int kRows = Stream::Slot::kRows;
  __shared__ typename Stream::Slot slots[WAVES];
  __shared__ float4_t sums[WAVES][TOKENS][4];  // 16 rows a token
  __shared__ int32_t ids[kMx4MoePairs];
  __shared__ uint16_t members[WAVES][TOKENS];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4, r0 = blockIdx.x * 16;
  for (int p = threadIdx.x; p < a.pairs; p += 64 * WAVES) ids[p] = a.ids[p];
  for (int i = lane; i < TOKENS * 4; i += 64) sums[wave][i / 4][i % 4] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  __syncthreads();
  const uint32_t blocks = a.inter_blocks;
  Stream st;
  st.slot = slots + wave;
  st.first = 0;
  st.end = blocks;
  st.plane = (uint32_t)a.pairs * blocks * 64u;
  st.xr = make_rsrc(a.h, (uint64_t)kMx4Planes * st.plane);
#pragma unroll
  for (int i = 0; i < 2; ++i) st.woff[i] = mx4_w_row(i, lane) * blocks * 16;
  st.column = r & (kRows - 1);
  int turn = 0;  // experts seen
  for (int base = 0; base < a.pairs; base += 64) {
    uint64_t todo = __ballot(base + lane < a.pairs && a.leads[min(base + lane, a.pairs - 1)] != 0);
    for (; todo != 0ull; todo &= todo - 1, ++turn) {
      if (turn % WAVES != wave) continue;
      const int e = __builtin_amdgcn_readfirstlane(ids[base + __builtin_ctzll(todo)]);
      int mine = -1;  // the pair of token `lane`
      for (int s = 0; s < a.top_k; ++s) {
        const int p = lane * a.top_k + s;
        if (lane < a.T && ids[p] == e) mine = p;
      }
      const uint64_t m = __ballot(mine >= 0);
      const int count = __popcll(m);
      if (mine >= 0) members[wave][__popcll(m & ((1ull << lane) - 1))] = (uint16_t)mine;
      wave_lds_fence();
      const int64_t row0 = (int64_t)e * a.hidden_blocks * 32 + r0;
      st.wr = make_rsrc(a.dn + row0 * blocks * 16, (uint64_t)16 * blocks * 16);
      const Mx4Scales ws(a.dns + row0 * blocks, 16 * blocks);
      st.wsr = ws.rsrc;
      st.wsoff = ws.word(mx4_s_row(lane) * blocks, lane);
      st.ws_skew = ws.skew(r * blocks);
      for (int m0 = 0; m0 < count; m0 += kRows) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const int row = m0 + mx4_x_row<kMx4XPlanes>(i, lane);
          st.xoff[i] = row < count ? (uint32_t)members[wave][row] * blocks * 64u : kOutOfRange;
        }
        const bool live = r < kRows && m0 + r < count;
        const int pair = live ? members[wave][m0 + r] : 0;
        const float f = a.weights[pair];
        float4_t acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
        st.run(acc, 0, 1, lane);
        if (live) {
          float4_t* s = &sums[wave][pair / a.top_k][g];
          const float4_t d = acc[0] + acc[1];
          float4_t o = *s;
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = fmaf(f, d[i], o[i]);
          *s = o;
        }
        wave_lds_fence();
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * 4; i += 64 * WAVES) {
    const int t = i / 4, q = i % 4;
    float4_t s = sums[0][t][q];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += sums[w][t][q];
    const float v[4] = {s[0], s[1], s[2], s[3]};
    store_run<4>(a.y, (int64_t)t * a.hidden_blocks * 32 + r0 + 4 * q, v, a.y_kind);
  }
}

template <int XK, int NL>
void run_up(const MoeArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.inter_blocks * 4, (unsigned)a.pairs);
  hipLaunchKernelGGL((vq_mx4_moe_up_kernel<XK, 4, NL, 3>), grid, dim3(256), 0, s, a);
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
  if (x_kind == kMx4XF16) T <= 4 ? run_up<kMx4XF16, 1>(a, s) : run_up<kMx4XF16, 2>(a, s);
  else T <= 4 ? run_up<kMx4XBF16, 1>(a, s) : run_up<kMx4XBF16, 2>(a, s);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)a.hidden_blocks * 2);
  if (T <= 16) hipLaunchKernelGGL((vq_mx4_moe_down_kernel<8, 1, 2, 16>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((vq_mx4_moe_down_kernel<8, 1, 2, 64>), grid, dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace vqmi
