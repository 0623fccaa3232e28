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
  uint16_t* h;     // [kMx4Planes][pairs][inter]
  int T, top_k, pairs, experts;
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

// The pairs of a call grouped by expert, in LDS: every block works them out for
// itself (about 1 us, less than another launch).
struct Groups {
  uint32_t first[kMx4MoeExperts];  // an expert's first pair
  uint16_t ids[kMx4MoePairs];      // kNone: no expert
  uint16_t leads[kMx4MoePairs];    // the experts' first pairs, in order
  int count;                       // of experts that are hit
  static constexpr uint16_t kNone = 0xffffu;
};

template <int THREADS>
__device__ __forceinline__ void group_pairs(Groups& s, const MoeArgs& a) {
  const bool one = a.T == 1;  // a token's experts are distinct
  for (int p = threadIdx.x; p < a.pairs; p += THREADS) s.ids[p] = (uint16_t)a.ids[p];
  if (!one) {
    for (int e = threadIdx.x; e < a.experts; e += THREADS) s.first[e] = ~0u;
    __syncthreads();
    for (int p = threadIdx.x; p < a.pairs; p += THREADS)
      if (s.ids[p] != Groups::kNone) atomicMin(&s.first[s.ids[p]], (uint32_t)p);
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int n = 0;
    for (int base = 0; base < a.pairs; base += 64) {
      const int p = base + lane;
      const uint16_t e = p < a.pairs ? s.ids[p] : Groups::kNone;
      const bool lead = e != Groups::kNone && (one || s.first[e] == (uint32_t)p);
      const uint64_t m = __ballot(lead);
      if (lead) s.leads[n + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)p;
      n += __popcll(m);
    }
    if (lane == 0) s.count = n;
  }
  __syncthreads();
}

// The pairs of expert e: lane t looks for token t's.  Writes them in the order
// of the tokens to `members` (the wave's own) and returns how many there are.
__device__ __forceinline__ int find_members(const Groups& s, const MoeArgs& a, int e, uint16_t* members, int lane) {
  int mine = -1;
  for (int k = 0; k < a.top_k; ++k) {
    const int p = lane * a.top_k + k;
    if (lane < a.T && s.ids[p] == e) mine = p;
  }
  const uint64_t m = __ballot(mine >= 0);
  wave_lds_fence();
  if (mine >= 0) members[__popcll(m & ((1ull << lane) - 1))] = (uint16_t)mine;
  wave_lds_fence();
  return __popcll(m);
}

// A wave's (or block's) work: 16 rows of an expert and up to kRows of its
// pairs.  `index` runs through experts (slowly) and tiles of rows (fast).
template <int NL>
struct MoeItem {
  Mx4Source<NL> src;
  int index, m0, count;  // count: the expert's pairs, m0: the first of them taken here
  int r0, pair;          // first row; the lane's column's pair, or -1
};

template <typename Stream, int NL>
__device__ __forceinline__ void set_item(MoeItem<NL>& it, int e, const uint8_t* w, const uint8_t* ws, int64_t row0,
                                         uint32_t blocks, const uint16_t* members, int top_k_or_one, int lane) {
  it.src.wr = make_rsrc(w + row0 * blocks * 16, (uint64_t)16 * blocks * 16);
  const Mx4Scales sc(ws + row0 * blocks, 16 * blocks);
  it.src.wsr = sc.rsrc;
  it.src.wsoff = sc.word(mx4_s_row(lane) * blocks, lane);
  it.src.ws_skew = sc.skew((lane & 15) * blocks);
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int row = it.m0 + mx4_x_row<kMx4XBF16>(i, lane);
    it.src.xoff[i] = row < it.count ? (uint32_t)(members[min(row, 63)] / top_k_or_one) * blocks * 64u : kOutOfRange;
  }
  const int c = lane & 15;
  it.pair = c < Stream::Slot::kRows && it.m0 + c < it.count ? members[min(it.m0 + c, 63)] : -1;
}

// No further work: loads of nothing.
template <int NL>
__device__ __forceinline__ void set_none(MoeItem<NL>& it, const void* any) {
  it.src.wr = it.src.wsr = make_rsrc(any, 0);
  it.src.wsoff = kOutOfRange;
  it.src.ws_skew = 0;
#pragma unroll
  for (int i = 0; i < NL; ++i) it.src.xoff[i] = kOutOfRange;
  it.pair = -1;
}

// Gate and up.  KW waves split the columns of an item (KW = 1: each wave has
// items of its own); the loads of the next item are under way while one is
// multiplied.
template <int XK, int KW, int NL, int DEPTH>
__global__ __launch_bounds__(256) void vq_mx4_moe_up_kernel(MoeArgs a) {
  typedef Mx4Stream<XK, 1, NL, DEPTH> Stream;
  constexpr int kRows = Stream::Slot::kRows, kWaves = 4;
  __shared__ typename Stream::Slot slots[kWaves];
  __shared__ float4_t part[KW > 1 ? kWaves : 1][64];
  __shared__ Groups groups;
  __shared__ uint16_t members[kWaves][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  group_pairs<64 * kWaves>(groups, a);
  const uint32_t blocks = a.hidden_blocks;
  const int tiles = a.inter_blocks * 4, items = __builtin_amdgcn_readfirstlane(groups.count) * tiles;
  const int stride = KW > 1 ? gridDim.x : gridDim.x * kWaves;
  Stream st;
  st.slot = slots + wave;
  st.first = 0;
  st.end = blocks;
  st.xr = make_rsrc(a.x, (uint64_t)a.T * blocks * 64);
  st.plane = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) st.woff[i] = mx4_w_row(i, lane) * blocks * 16;
  st.column = r & (kRows - 1);
  auto set = [&](MoeItem<NL>& it) VQMI_INLINE {  // at it.index, its pairs from it.m0 on (0: to be found)
    if (it.index >= items) return set_none(it, a.x);
    const int e = __builtin_amdgcn_readfirstlane(groups.ids[groups.leads[it.index / tiles]]);
    if (it.m0 == 0) it.count = find_members(groups, a, e, members[wave], lane);
    it.r0 = it.index % tiles * 16;
    set_item<Stream>(it, e, a.gu, a.gus, (int64_t)e * a.inter_blocks * 64 + it.r0, blocks, members[wave], a.top_k, lane);
  };
  MoeItem<NL> cur, next;
  cur.index = KW > 1 ? blockIdx.x : blockIdx.x * kWaves + wave;
  cur.m0 = cur.count = 0;
  set(cur);
  const uint32_t from = KW > 1 ? wave : 0;
  st.start(cur.src, from, KW, lane);
  while (cur.index < items) {
    next.index = cur.index;
    next.count = cur.count;
    next.m0 = cur.m0 + kRows;
    if (next.m0 >= cur.count) next.index += stride, next.m0 = 0;
    set(next);
    float4_t acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    st.run(acc, cur.src, next.src, from, KW, lane);
    float4_t s = acc[0] + acc[1];
    if constexpr (KW > 1) {
      part[wave][lane] = s;
      lds_barrier();
      s = part[0][lane];
#pragma unroll
      for (int w = 1; w < KW; ++w) s += part[w][lane];
      lds_barrier();
    }
    if ((KW == 1 || wave == 0) && cur.pair >= 0) {
      uint32_t lo[kMx4Planes], hi[kMx4Planes];
      split_planes(silu_mul<true>(s[0], s[1]), lo);
      split_planes(silu_mul<true>(s[2], s[3]), hi);
      const int64_t inter = (int64_t)a.inter_blocks * 32;
      uint16_t* out = a.h + cur.pair * inter + cur.r0 / 2 + 2 * g;
#pragma unroll
      for (int p = 0; p < kMx4Planes; ++p)
        *reinterpret_cast<uint32_t*>(out + p * a.pairs * inter) = lo[p] | hi[p] << 16;
    }
    cur = next;
  }
}

// Down: a block takes 16 output rows for all tokens, its waves the experts in
// turn, for the pairs of an expert, kRows at a time.  A wave adds up its
// experts' weighted products per token in LDS, in the order of the experts; the
// waves' sums are joined in their order.
template <int WAVES, int NL, int DEPTH, int TOKENS>
__global__ __launch_bounds__(64 * WAVES) void vq_mx4_moe_down_kernel(MoeArgs a) {
  typedef Mx4Stream<kMx4XPlanes, kMx4Planes, NL, DEPTH> Stream;
  constexpr int kRows = Stream::Slot::kRows;
  __shared__ typename Stream::Slot slots[WAVES];
  __shared__ float4_t sums[WAVES][TOKENS][4];  // 16 rows a token
  __shared__ Groups groups;
  __shared__ uint16_t members[WAVES][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4, r0 = blockIdx.x * 16;
  for (int i = lane; i < TOKENS * 4; i += 64) sums[wave][i / 4][i % 4] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  group_pairs<64 * WAVES>(groups, a);
  const uint32_t blocks = a.inter_blocks;
  const int items = __builtin_amdgcn_readfirstlane(groups.count);
  Stream st;
  st.slot = slots + wave;
  st.first = 0;
  st.end = blocks;
  st.plane = (uint32_t)a.pairs * blocks * 64u;
  st.xr = make_rsrc(a.h, (uint64_t)kMx4Planes * st.plane);
#pragma unroll
  for (int i = 0; i < 2; ++i) st.woff[i] = mx4_w_row(i, lane) * blocks * 16;
  st.column = r & (kRows - 1);
  float weight_next = 0.0f;
  auto set = [&](MoeItem<NL>& it) VQMI_INLINE {
    if (it.index >= items) return set_none(it, a.h);
    const int e = __builtin_amdgcn_readfirstlane(groups.ids[groups.leads[it.index]]);
    if (it.m0 == 0) it.count = find_members(groups, a, e, members[wave], lane);
    set_item<Stream>(it, e, a.dn, a.dns, (int64_t)e * a.hidden_blocks * 32 + r0, blocks, members[wave], 1, lane);
    weight_next = a.weights[max(it.pair, 0)];
  };
  MoeItem<NL> cur, next;
  cur.index = wave;
  cur.m0 = cur.count = 0;
  set(cur);
  st.start(cur.src, 0, 1, lane);
  while (cur.index < items) {
    const float f = weight_next;
    next.index = cur.index;
    next.count = cur.count;
    next.m0 = cur.m0 + kRows;
    if (next.m0 >= cur.count) next.index += WAVES, next.m0 = 0;
    set(next);
    float4_t acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    st.run(acc, cur.src, next.src, 0, 1, lane);
    if (cur.pair >= 0) {
      float4_t* s = &sums[wave][cur.pair / a.top_k][g];
      const float4_t d = acc[0] + acc[1];
      float4_t o = *s;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(f, d[i], o[i]);
      *s = o;
    }
    wave_lds_fence();
    cur = next;
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

template <int XK>
void run_up(const MoeArgs& a, hipStream_t s) {
  const int tiles = a.inter_blocks * 4, most = min(a.pairs, a.experts) * tiles;  // items at most
  if (a.T <= 2) {
    hipLaunchKernelGGL((vq_mx4_moe_up_kernel<XK, 4, 1, 2>), dim3(min(most, 1 << 16)), dim3(256), 0, s, a);
  } else {
    hipLaunchKernelGGL((vq_mx4_moe_up_kernel<XK, 1, 1, 2>), dim3(min((most + 3) / 4, 1024)), dim3(256), 0, s, a);
  }
}

}  // namespace

size_t mx4_moe_workspace_bytes(int T, int top_k, int inter) {
  return kMx4Planes * (size_t)T * top_k * inter * sizeof(uint16_t);
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
  a.experts = r.num_experts;
  a.h = static_cast<uint16_t*>(workspace);
  a.hidden_blocks = gate_up.cols / kMx4Block;
  a.inter_blocks = down.cols / kMx4Block;
  a.y_kind = y_kind;
  if (x_kind == kMx4XF16) run_up<kMx4XF16>(a, s);
  else run_up<kMx4XBF16>(a, s);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)a.hidden_blocks * 2);
  if (T <= 16) hipLaunchKernelGGL((vq_mx4_moe_down_kernel<8, 1, 2, 16>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((vq_mx4_moe_down_kernel<8, 1, 2, 64>), grid, dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace vqmi
