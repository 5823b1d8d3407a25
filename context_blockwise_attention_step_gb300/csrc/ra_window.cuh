// ra_window.cuh — warp-collective walks of the windowed kernels over a block's tiles.
//
// A windowed block sees tiles of few shards, and finding a shard's tiles takes a chain of
// layout arithmetic (~200 cycles): a warp works out 32 shards at once, one per lane, and walks
// the shards that have tiles.
#pragma once
#include "ra_plan.h"

namespace ra {

// Calls body(i, tiles) for every i in [0, n) whose set is not empty, in order, with the whole
// warp; stops when body returns false (body's answer must be the same in all lanes). Returns
// false if stopped.
template <typename SetF, typename BodyF>
__device__ __forceinline__ bool for_each_set(int n, SetF&& set, BodyF&& body) {
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < n; base += 32) {
    TileSet t = {0, 0, 0, 0, 0};
    if (base + lane < n) t = set(base + lane);
    unsigned left = __ballot_sync(0xffffffffu, tile_count(t) > 0);
    while (left != 0) {
      const int src = __ffs(left) - 1;
      left &= left - 1;
      TileSet u;
      u.sink = __shfl_sync(0xffffffffu, t.sink, src);
      u.s0 = __shfl_sync(0xffffffffu, t.s0, src);
      u.n0 = __shfl_sync(0xffffffffu, t.n0, src);
      u.s1 = __shfl_sync(0xffffffffu, t.s1, src);
      u.n1 = __shfl_sync(0xffffffffu, t.n1, src);
      if (!body(base + src, u)) return false;
    }
  }
  return true;
}

// Bit i: set(base + i) is not empty, for the 32 sets from base on.
template <typename SetF>
__device__ __forceinline__ unsigned nonempty(int n, int base, SetF&& set) {
  const int i = base + (threadIdx.x & 31);
  return __ballot_sync(0xffffffffu, i < n && tile_count(set(i)) > 0);
}

// The tiles of all n sets.
template <typename SetF>
__device__ __forceinline__ int count_tiles(int n, SetF&& set) {
  int c = 0;
  for (int i = threadIdx.x & 31; i < n; i += 32) c += tile_count(set(i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
  return c;
}

// Bits 0 .. n-1 set, n clamped to [0, 32].
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// The visible columns c of a tile among [cs, cs + 32): c < cnt and (c >= lo or c < sk).
__device__ __forceinline__ uint32_t visible_bits(int cs, int cnt, int lo, int sk) {
  return low_bits(cnt - cs) & (~low_bits(lo - cs) | low_bits(sk - cs));
}

}  // namespace ra
