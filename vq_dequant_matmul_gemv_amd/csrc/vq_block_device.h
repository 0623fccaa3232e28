// vq_block_device.h -- device code that the kernels of the operators around the
// products share.
#pragma once

#include "vq_device.h"

#include <type_traits>
#include <utility>

namespace vqmi {

// f(0), ..., f(N - 1) with the index as a constant: a loop whose body is chosen
// by it is unrolled whatever its size.
template <typename F, int... I>
__device__ __forceinline__ void static_for_each(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_each(static_cast<F&&>(f), std::make_integer_sequence<int, N>{});
}
#define VQMI_INLINE __attribute__((always_inline))

// One wave's LDS writes before its later reads of other lanes' values (LDS
// runs a wave's accesses in order: only the compiler is held back).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The tile of output rows and tokens that a block takes, XCD-aware: blocks land
// on XCD (block % 8); each XCD takes a contiguous range of tiles, which run
// through up to 8 token tiles of one row tile before the next.
__device__ __forceinline__ void xcd_tile(int block, int row_tiles, int tok_tiles, int* row_tile, int* tok_tile) {
  const int n = row_tiles * tok_tiles, q = n / 8, r8 = n % 8, xcd = block % 8, j = block / 8;
  const int tile = xcd * q + min(xcd, r8) + j;
  const int g = tile / (8 * row_tiles), rem = tile - g * 8 * row_tiles, width = min(8, tok_tiles - 8 * g);
  *row_tile = rem / width;
  *tok_tile = 8 * g + rem % width;
}

}  // namespace vqmi
