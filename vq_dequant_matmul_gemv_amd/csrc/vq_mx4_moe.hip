// vq_mx4_moe.hip -- a mixture-of-experts layer for a few tokens over 4-bit
// experts: one kernel for the gate and up projections with SwiGLU (and, up to 5
// tokens, the routing) and one for the down projection with the weighted sum
// (where many tokens share experts, the sum in a third).
//
//   h[t][s] = silu(W_gate[e] x_t) * (W_up[e] x_t),   e = ids[t][s]
//   y[t]    = sum over the slots s of weight[t][s] * W_down[e] h[t][s]
//
// Bound by the bytes of the experts that the tokens hit, so an expert's weights
// are read once for a group of the pairs (token and slot) that chose it, which
// are the columns of its matrix products.  256 experts, top 8, of 4096 x 1024:
// 64 tokens that hit 182 of them (1.2 GB) take 277 to 295 us, 16 that hit 90 136
// to 141, 4.1 to 4.4 TB/s of a copy's 5.2; one token (53 MB) 21.5 us: 12 of gate and up
// with the routing, 8 of down, each launch's latency and ramp beside 7 and 3.5
// us of bytes.
//
// h is kept in fp32 as three bf16 planes, so that the down products take it
// whole: rounding it to 16 bits would add an error that the caller's sums of
// 16-bit products do not have.
#include "vq_block_kernels.h"
#include "vq_mx4_device.h"
#include "vq_mx4_groups.h"
#include "vq_router_device.h"
#include "vq_store_device.h"

namespace vqmi {

namespace {

struct MoeArgs {
  const uint8_t *gu, *gus, *dn, *dns;  // gate and up rows in turn, down: values and scales
  const void* x;
  void* y;
  const int32_t* ids;
  const float* weights;
  uint16_t* h;      // [kMx4Planes][pairs][inter]
  float* products;  // [pairs][hidden]
  int T, top_k, pairs, experts;
  int hidden_blocks, inter_blocks;  // blocks of 32 columns
  int y_kind;
  RouterArgs route;  // of the kernels that route their own tokens
  int route_kind;
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

// The pairs of a call in groups of one expert's, at most kRows each, in LDS:
// every block works them out for itself (1 to 2 us, less than another launch).
struct Groups {
  uint16_t expert[kMx4MoePairs], start[kMx4MoePairs + 1];  // a group's expert, and where its pairs start
  uint16_t pair[kMx4MoePairs];                             // by expert, then by token
  uint8_t token[kMx4MoePairs];
  int count;                                               // of groups
};
struct GroupScratch {                // while they are worked out
  uint32_t mask[2][kMx4MoeExperts];  // the tokens that chose an expert
  uint16_t at[kMx4MoeExperts];       // where an expert's pairs start in `pair`
};

// The sum of v over the lanes up to this one: within rows of 16 by shifts, then
// the rows before by their last lanes.
__device__ __forceinline__ uint32_t lanes_sum_up_to(uint32_t v) {
#define VQMI_ADD(ctrl, rows) v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false)
  VQMI_ADD(0x111, 0xf);
  VQMI_ADD(0x112, 0xf);
  VQMI_ADD(0x114, 0xf);
  VQMI_ADD(0x118, 0xf);
  VQMI_ADD(0x142, 0xa);
  VQMI_ADD(0x143, 0xc);
#undef VQMI_ADD
  return v;
}

// The routing of up to 5 tokens by each block of 4 waves, the way a launch of
// its own would, for the shapes (lanes of a token, experts of a lane) that
// routers of up to 256 experts commonly have.  Saves that launch, less what the
// blocks take: 24.0 -> 22.5 us with 256 experts top 8 of 4096x1024 and one
// token, 11.5 -> 10.1 with 60 top 4 of 1504x352.  Up to 5 tokens: those of the
// kernel with groups of 2 pairs.  The kernel with groups of 4 would gain as much
// with a copy of its own (256 top 8 of 4096x1024 at 6 tokens 67.2 -> 65.1, 8 78.9
// -> 77.5; 60 top 4 of 1504x352 at 6 18.0 -> 16.7, 16 24.0 -> 22.7; 8 top 2 of
// 1024x512 at 8 13.3 -> 11.9), which is not built.
constexpr int kRouteTokens = 5, kRoutePairs = kRouteTokens * 32;
struct RouteScratch {
  double wave[4][kRouteLds<32, 8>];
};
int route_kind(const RouterPlan& p, int logits_kind) {  // -1: none of these
  if (p.lanes != 16 && !(p.lanes == 32 && p.per_lane == 8)) return -1;
  const int shape = p.lanes == 32 ? 4 : p.per_lane == 1 ? 0 : p.per_lane == 2 ? 1 : p.per_lane == 4 ? 2 : 3;
  return 3 * shape + (logits_kind == kOutF32 ? 0 : logits_kind == kOutF16 ? 1 : 2);
}
__device__ __forceinline__ void route_tokens(const RouterArgs& r, int kind, RouteScratch& x, int wave, int lane) {
  const int per = kind < 12 ? 4 : 2, t0 = wave * per;  // tokens a wave
  if (t0 >= r.T) return;
#define VQMI_ROUTE(k, lanes, experts)                                                   \
  case 3 * k: return route_wave<lanes, experts, kOutF32>(r, x.wave[wave], t0, lane);     \
  case 3 * k + 1: return route_wave<lanes, experts, kOutF16>(r, x.wave[wave], t0, lane); \
  case 3 * k + 2: return route_wave<lanes, experts, kOutBF16>(r, x.wave[wave], t0, lane);
  switch (kind) {
    VQMI_ROUTE(0, 16, 1)
    VQMI_ROUTE(1, 16, 2)
    VQMI_ROUTE(2, 16, 4)
    VQMI_ROUTE(3, 16, 8)
    VQMI_ROUTE(4, 32, 8)
  }
#undef VQMI_ROUTE
}

template <int THREADS, int ROWS>
__device__ __forceinline__ void group_pairs(Groups& s, GroupScratch& x, const MoeArgs& a, const int32_t* ids) {
  constexpr int kPer = kMx4MoePairs / THREADS;
  const int lane = threadIdx.x & 63;
  if (a.T == 1) {  // a token's experts are distinct
    if (threadIdx.x < 64) {
      const int e = lane < a.pairs ? ids[lane] : -1;
      const uint64_t m = __ballot(e >= 0);
      const int i = __popcll(m & ((1ull << lane) - 1)), n = __popcll(m);
      if (e >= 0) {
        s.expert[i] = (uint16_t)e;
        s.pair[i] = (uint16_t)lane;
        s.token[i] = 0;
      }
      s.start[lane] = (uint16_t)lane;
      if (lane == 0) s.start[64] = 64, s.count = n;
    }
    __syncthreads();
    return;
  }
  int e[kPer], t[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = threadIdx.x + i * THREADS;
    e[i] = p < a.pairs ? ids[p] : -1;
    t[i] = p / a.top_k;
  }
  for (int k = threadIdx.x; k < a.experts; k += THREADS) x.mask[0][k] = x.mask[1][k] = 0u;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (e[i] >= 0) atomicOr(&x.mask[t[i] >> 5][e[i]], 1u << (t[i] & 31));
  __syncthreads();
  if (threadIdx.x < 64) {
    uint32_t before = 0;  // pairs, and groups in the upper half
    for (int base = 0; base < a.experts; base += 64) {
      const int k = base + lane;
      const uint32_t c = k < a.experts ? __popc(x.mask[0][k]) + __popc(x.mask[1][k]) : 0;
      const uint32_t both = c | (c + ROWS - 1) / ROWS << 16, sum = lanes_sum_up_to(both), at = before + sum - both;
      if (c > 0) x.at[k] = (uint16_t)at;
      for (uint32_t m = 0; m < c; m += ROWS) {
        s.expert[(at >> 16) + m / ROWS] = (uint16_t)k;
        s.start[(at >> 16) + m / ROWS] = (uint16_t)(at + m);
      }
      before += (uint32_t)__builtin_amdgcn_readlane((int)sum, 63);
    }
    if (lane == 0) s.start[before >> 16] = (uint16_t)before, s.count = before >> 16;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (e[i] < 0) continue;
    const uint32_t below = (1u << (t[i] & 31)) - 1u, lo = x.mask[0][e[i]], hi = x.mask[1][e[i]];
    const int at = x.at[e[i]] + (t[i] < 32 ? __popc(lo & below) : __popc(lo) + __popc(hi & below));
    s.pair[at] = (uint16_t)(threadIdx.x + i * THREADS);
    s.token[at] = (uint8_t)t[i];
  }
  __syncthreads();
}

// A wave's (or block's) work: 16 * MT rows of a group's expert and its pairs.
template <int MT, int NL>
struct MoeItem {
  Mx4Source<MT, NL> src;
  int group, tile;  // which group, which rows
  int pair;         // of the column that the lane multiplies, or -1

  // (member by member: as a whole the compiler copies it through memory, and
  // waits for every load in flight)
  __device__ __forceinline__ void take(const MoeItem& o) {
    src.take(o.src);
    group = o.group, tile = o.tile, pair = o.pair;
  }
};

// Gate and up (UP: 16-bit activations, SwiGLU, h out) or down (h in, the pairs'
// products out).  KW waves split the columns of an item (KW = 1: each wave has
// items of its own); the loads of the next item are under way while one is
// multiplied.  ROUTE: every block routes the call's few tokens for itself, one
// of them for the outputs.
template <int XK, int KW, int MT, int NL, int DEPTH, int PER_CU, bool ROUTE>
__global__ __launch_bounds__(256, PER_CU) void vq_mx4_moe_kernel(MoeArgs a) {
  constexpr bool kUp = XK != kMx4XPlanes;
  typedef Mx4Stream<XK, kUp ? 1 : kMx4Planes, MT, NL, DEPTH> Stream;
  constexpr int kRows = Stream::Slot::kRows, kWaves = 4;
  __shared__ union {
    typename Stream::Slot slots[kWaves];
    GroupScratch scratch;
    RouteScratch route;
  } lds;
  __shared__ float4_t part[KW > 1 ? kWaves : 1][MT][64];
  __shared__ Groups groups;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  __shared__ int32_t ids[ROUTE ? kRoutePairs : 1];
  __shared__ float weights[ROUTE ? kRoutePairs : 1];
  if constexpr (ROUTE) {
    RouterArgs route = a.route;
    route.ids = ids;
    route.weights = weights;
    route_tokens(route, a.route_kind, lds.route, wave, lane);
    __syncthreads();
  }
  group_pairs<64 * kWaves, kRows>(groups, lds.scratch, a, ROUTE ? ids : a.ids);
  const int count = __builtin_amdgcn_readfirstlane(groups.count);
  const uint32_t blocks = kUp ? a.hidden_blocks : a.inter_blocks;
  const int tiles = (kUp ? a.inter_blocks * 4 : a.hidden_blocks * 2) / MT;
  const int units = KW > 1 ? gridDim.x : gridDim.x * kWaves;  // that share the items
  const int step_group = units / tiles, step_tile = units % tiles;
  const uint8_t *w = kUp ? a.gu : a.dn, *ws = kUp ? a.gus : a.dns;
  Stream st;
  st.slot = lds.slots + wave;
  st.first = 0;
  st.end = blocks;
  st.plane = kUp ? 0u : (uint32_t)a.pairs * blocks * 64u;
  st.xr = kUp ? make_rsrc(a.x, (uint64_t)a.T * blocks * 64) : make_rsrc(a.h, (uint64_t)kMx4Planes * st.plane);
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) st.woff[i] = mx4_w_row(i, lane) * blocks * 16;
  st.column = r & (kRows - 1);
  auto set = [&](MoeItem<MT, NL>& it) VQMI_INLINE {
    if (it.group >= count) return it.src.clear();  // no further work
    const int e = __builtin_amdgcn_readfirstlane(groups.expert[it.group]);
    const int first = groups.start[it.group], last = groups.start[it.group + 1] - 1;
    const int64_t row0 = ((int64_t)e * tiles + it.tile) * (16 * MT);
    it.src.w = w + row0 * blocks * 16;
    it.src.w_bytes = 16 * MT * blocks * 16;
    const Mx4Scales sc(ws + row0 * blocks, 16 * MT * blocks);
    it.src.ws = sc.base;
    it.src.ws_bytes = sc.bytes;
#pragma unroll
    for (int i = 0; i < MT; ++i) it.src.wsoff[i] = sc.place(mx4_s_row(i, lane) * blocks, lane);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int p = first + mx4_x_row<XK>(i, lane), q = min(p, last);
      const uint32_t row = kUp ? groups.token[q] : groups.pair[q];
      it.src.xoff[i] = p <= last ? row * blocks * 64u : kOutOfRange;
    }
    const int pair = groups.pair[min(first + r, last)];
    it.pair = first + r <= last ? pair : -1;
  };
  MoeItem<MT, NL> cur, next;
  const int unit = KW > 1 ? blockIdx.x : blockIdx.x * kWaves + wave;
  cur.group = unit / tiles;
  cur.tile = unit % tiles;
  cur.pair = -1;
  cur.src.w = cur.src.ws = w;
#pragma unroll
  for (int i = 0; i < MT; ++i) cur.src.wsoff[i] = kOutOfRange;
  set(cur);
  const uint32_t from = KW > 1 ? wave : 0;
  st.start(cur.src, from, KW, lane);
  while (cur.group < count) {
    next.take(cur);
    next.group += step_group;
    next.tile += step_tile;
    if (next.tile >= tiles) next.tile -= tiles, next.group += 1;
    set(next);
    float4_t acc[MT][2], s[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    st.run(acc, cur.src, next.src, from, KW, lane);
#pragma unroll
    for (int m = 0; m < MT; ++m) s[m] = acc[m][0] + acc[m][1];
    if constexpr (KW > 1) {
#pragma unroll
      for (int m = 0; m < MT; ++m) part[wave][m][lane] = s[m];
      lds_barrier();
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        s[m] = part[0][m][lane];
#pragma unroll
        for (int k = 1; k < KW; ++k) s[m] += part[k][m][lane];
      }
      lds_barrier();
    }
    if ((KW == 1 || wave == 0) && cur.pair >= 0) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int r0 = (cur.tile * MT + m) * 16;
        if constexpr (kUp) {
          uint32_t lo[kMx4Planes], hi[kMx4Planes];
          split_planes(silu_mul<true>(s[m][0], s[m][1]), lo);
          split_planes(silu_mul<true>(s[m][2], s[m][3]), hi);
          const int64_t inter = (int64_t)a.inter_blocks * 32;
          uint16_t* out = a.h + cur.pair * inter + r0 / 2 + 2 * g;
#pragma unroll
          for (int p = 0; p < kMx4Planes; ++p)
            *reinterpret_cast<uint32_t*>(out + p * a.pairs * inter) = lo[p] | hi[p] << 16;
        } else {
          *reinterpret_cast<float4_t*>(a.products + ((int64_t)cur.pair * a.hidden_blocks * 32 + r0 + 4 * g)) = s[m];
        }
      }
    }
    cur.take(next);
  }
  if constexpr (ROUTE) {
    if (blockIdx.x == 0 && (int)threadIdx.x < a.pairs) {
      a.route.ids[threadIdx.x] = ids[threadIdx.x];
      a.route.weights[threadIdx.x] = weights[threadIdx.x];
    }
  }
}

// The pairs' products, weighted, in the order of the slots: 4 columns a thread.
__global__ __launch_bounds__(256) void vq_mx4_moe_sum_kernel(MoeArgs a) {
  const int per = a.hidden_blocks * 8, i = blockIdx.x * 256 + threadIdx.x, t = i / per, c = i % per * 4;
  if (t >= a.T) return;
  float4_t y = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = 0; s0 < a.top_k; s0 += 8) {
    float4_t v[8];  // eight slots in flight
    float f[8];
    bool live[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int p = t * a.top_k + min(s0 + s, a.top_k - 1);
      live[s] = s0 + s < a.top_k && a.ids[p] >= 0;
      f[s] = a.weights[p];
      v[s] = *reinterpret_cast<const float4_t*>(a.products + (int64_t)p * a.hidden_blocks * 32 + c);
    }
#pragma unroll
    for (int s = 0; s < 8; ++s) {
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = live[s] ? fmaf(f[s], v[s][k], y[k]) : y[k];
    }
  }
  const float v[4] = {y[0], y[1], y[2], y[3]};
  store_run<4>(a.y, (int64_t)t * a.hidden_blocks * 32 + c, v, a.y_kind);
}

// Down for a token or two: a block takes 16 output rows, its waves the pairs in
// turn; their weighted products are joined in the order of the waves.
template <int WAVES, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void vq_mx4_moe_down_kernel(MoeArgs a) {
  typedef Mx4Stream<kMx4XPlanes, kMx4Planes, 1, 1, DEPTH> Stream;
  __shared__ typename Stream::Slot slots[WAVES];
  __shared__ float4_t part[WAVES][4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4, r0 = blockIdx.x * 16, t = blockIdx.y;
  const uint32_t blocks = a.inter_blocks;
  Stream st;
  st.slot = slots + wave;
  st.first = 0;
  st.end = blocks;
  st.plane = (uint32_t)a.pairs * blocks * 64u;
  st.xr = make_rsrc(a.h, (uint64_t)kMx4Planes * st.plane);
#pragma unroll
  for (int i = 0; i < 2; ++i) st.woff[i] = mx4_w_row(i, lane) * blocks * 16;
  st.column = 0;
  float f_next = 0.0f;
  auto set = [&](Mx4Source<1, 1>& src, int s) VQMI_INLINE {  // slot s of the token
    const int p = t * a.top_k + s, e = s < a.top_k ? __builtin_amdgcn_readfirstlane(a.ids[p]) : -1;
    f_next = 0.0f;
    if (e < 0) {
      src.w = src.ws = a.dn;
      src.wsoff[0] = kOutOfRange;
      src.clear();
      return;
    }
    const int64_t row0 = (int64_t)e * a.hidden_blocks * 32 + r0;
    src.w = a.dn + row0 * blocks * 16;
    src.w_bytes = 16 * blocks * 16;
    const Mx4Scales sc(a.dns + row0 * blocks, 16 * blocks);
    src.ws = sc.base;
    src.ws_bytes = sc.bytes;
    src.wsoff[0] = sc.place(mx4_s_row(0, lane) * blocks, lane);
    src.xoff[0] = mx4_x_row<kMx4XPlanes>(0, lane) == 0 ? (uint32_t)p * blocks * 64u : kOutOfRange;
    f_next = a.weights[p];
  };
  Mx4Source<1, 1> cur, next;
  set(cur, wave);
  st.start(cur, 0, 1, lane);
  float4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = wave; s < a.top_k; s += WAVES) {
    const float f = f_next;
    set(next, s + WAVES);
    float4_t acc[1][2] = {{{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}}};
    st.run(acc, cur, next, 0, 1, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = fmaf(f, acc[0][0][i] + acc[0][1][i], sum[i]);
    cur.take(next);
  }
  if (r == 0) part[wave][g] = sum;
  __syncthreads();
  if (threadIdx.x >= 4) return;
  float4_t y = part[0][threadIdx.x];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) y += part[w][threadIdx.x];
  const float v[4] = {y[0], y[1], y[2], y[3]};
  store_run<4>(a.y, (int64_t)t * a.hidden_blocks * 32 + r0 + 4 * threadIdx.x, v, a.y_kind);
}

// Down by each token's pairs on their own, without the launch that sums: saves
// 4 to 5 us and reads an expert again for each further token that chose it.
// The measured difference is m * (pairs / 20 + again / 3) us less those, for
// matrices of m MB of which chance has `again` read again.  us, groups -> on
// their own: 256 experts top 8 of 4096x1024 at 3 tokens 46.0 -> 41.1, 5 58.3 ->
// 57.5, 16 118 -> 140; of 2048x512 at 3 25.8 -> 20.5, 8 37.2 -> 33.6, 12 42.7
// -> 41.2, 16 44.7 -> 48.1; 60 top 4 of 1504x352 at 5 18.4 -> 14.4, 16 24.2 ->
// 24.6; 8 top 2 of 4096x1792 at 3 25.5 -> 25.8, 4 27.4 -> 30.0; 2 top 1 of
// 1024x512 at 16 16.3 -> 15.0, 32 17.2 -> 22.4.  Over 13 layers of 2 to 256
// experts at 2 to 64 tokens the choice takes 0.7 % longer than the better one on
// average, 15 % at worst (64 top 6 of 2048x1408 at 4: 35.8 -> 31.0, not taken).
// (A single token has no room for the products in its workspace.)
bool down_by_token(const MoeArgs& a) {
  const float m = 32.0f * 17.0f * a.hidden_blocks * a.inter_blocks * 1e-6f;
  const float again = 0.5f * a.T * (a.T - 1) * a.top_k * a.top_k / a.experts;
  return a.T == 1 || m * (a.pairs / 20.0f + again / 3.0f) < 3.5f;
}

// PER_CU: blocks that a compute unit holds, so that all of a launch run at once.
// As many of them as the pairs can make items: where tokens share few experts
// those are many more than experts * tiles, as many blocks as that leave most of
// the card idle (us, blocks for that -> for the groups: 2 experts top 1 of
// 1024x512 at 64 tokens 44.9 -> 18.7; 8 top 2 of 1024x512 at 16 20.3 -> 17.8, at
// 64 32.0 -> 22.6; 8 top 2 of 4096x1792 at 64 89.7 -> 80.3).
template <int XK, int KW, int MT, int NL, int DEPTH, int PER_CU, bool ROUTE = false>
void run_products(const MoeArgs& a, int tiles, hipStream_t s) {
  constexpr int kGroup = Mx4Slot<XK, 1, MT, NL>::kRows;
  const int items = mx4_moe_max_groups(a.pairs, a.experts, kGroup) * (tiles / MT);
  const int grid = min(KW > 1 ? items : (items + 3) / 4, 256 * PER_CU);
  hipLaunchKernelGGL((vq_mx4_moe_kernel<XK, KW, MT, NL, DEPTH, PER_CU, ROUTE>), dim3(grid), dim3(256), 0, s, a);
}

template <int XK>
hipError_t run_layer(const MoeArgs& a, hipStream_t s) {
  const int up = a.inter_blocks * 4, down = a.hidden_blocks * 2;
  // Gate and up by blocks that split the columns, with groups of 2 or 4 pairs,
  // or by waves on their own with twice the rows and groups of 8.  The groups
  // of 2 load least beside the weights (up to 5 tokens); waves on their own
  // need 1200 items or so to fill the card (2048 of them run at once), and gain
  // where most experts are chosen more than once.  us of the layer, groups of
  // 4 and 8 (and their items): 8 top 2 of 4096x1792 at 8 tokens 31.7 and 34.6
  // (1008), at 16 40.8 and 39.7 (1232), at 32 53.4 and 54.5 (1680), at 64 79.0
  // and 70.3 (2240); 32 top 4 of 1024x512 at 8 15.7 and 16.1 (1024), at 64 31.9
  // and 26.7 (1920); 4 top 2 of 2048x1024 at 16 21.7 and 23.8 (448), at 64 34.6
  // and 31.8 (1216); 60 top 4 of 1504x352 at 16 24.1 and 25.2 (1331), at 32 28.3
  // and 27.5 (1452); 256 top 8 of 4096x1024 at 16 117.9 and 119.9 (pairs <
  // experts), at 32 173 and 166 (16384), at 64 269 and 244.  Over 13 layers of 2
  // to 256 experts at 6 to 64 tokens the choice takes 0.4 % longer than the
  // better one on average, 9 % at worst (8 top 2 of 1024x512 at 64: 736 items,
  // 22.8 and 20.9).  Groups of 2 and 4 with 256 top 8 of 4096x1024: at 2 tokens
  // 31.8 and 32.6, at 5 58.8 and 59.4, at 8 79.7 and 79.4, at 16 122 and 118.
  const int eights = mx4_moe_max_groups(a.pairs, a.experts, 8) * (up / 2);
  if (a.route_kind >= 0) run_products<XK, 4, 1, 1, 2, 4, true>(a, up, s);
  else if (a.T <= kRouteTokens) run_products<XK, 4, 1, 1, 2, 4>(a, up, s);
  else if (a.pairs < a.experts || eights < 1200) run_products<XK, 4, 1, 2, 2, 4>(a, up, s);
  else run_products<XK, 1, 2, 4, 2, 2>(a, up, s);
  if (down_by_token(a)) {
    hipLaunchKernelGGL((vq_mx4_moe_down_kernel<8, 2>), dim3(down, a.T), dim3(512), 0, s, a);
  } else {
    run_products<kMx4XPlanes, 1, 2, 2, 1, 3>(a, down, s);
    hipLaunchKernelGGL(vq_mx4_moe_sum_kernel, dim3((a.T * a.hidden_blocks * 8 + 255) / 256), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

size_t mx4_moe_workspace_bytes(int T, int top_k, int hidden, int inter) {
  const size_t pairs = (size_t)T * top_k;
  return kMx4Planes * pairs * inter * sizeof(uint16_t) + (T == 1 ? 0 : pairs * hidden * sizeof(float));
}

hipError_t launch_mx4_moe(const RouterSpec& r, const Mx4View& gate_up, const Mx4View& down, const void* logits,
                          const void* x, int x_kind, int T, void* y, int y_kind, int32_t* ids, float* weights,
                          void* workspace, hipStream_t s) {
  const RouterPlan plan = router_plan(r, logits, T, ids, weights);
  MoeArgs a{};
  a.route = plan.args;
  a.route_kind = T <= kRouteTokens ? route_kind(plan, r.logits_kind) : -1;
  if (a.route_kind < 0) {
    const hipError_t e = launch_router(r, logits, T, ids, weights, s);
    if (e != hipSuccess) return e;
  }
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
  a.products = reinterpret_cast<float*>(a.h + (size_t)kMx4Planes * a.pairs * down.cols);
  return x_kind == kMx4XF16 ? run_layer<kMx4XF16>(a, s) : run_layer<kMx4XBF16>(a, s);
}

}  // namespace vqmi
