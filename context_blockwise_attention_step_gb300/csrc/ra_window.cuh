// ra_window.cuh — the windowed kernels' walks over a block's tiles.
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

// key_limit() for one position and many shards, in 32 bits (positions stay below 2^31): the
// stripe layout's division is done once.
struct KeyLimit {
  int p, d, m;  // position; p / D and p % D (stripe)
};
__device__ __forceinline__ KeyLimit key_limit_of(const Plan& P, int p) {
  KeyLimit k = {p, 0, 0};
  if (P.layout == kStripe && p >= 0) {
    k.d = p / P.D;
    k.m = p - k.d * P.D;
  }
  return k;
}
__device__ __forceinline__ int limit_in(const Plan& P, int L, int j, const KeyLimit& k) {
  if (k.p < 0) return -1;
  int b;
  if (P.layout == kStripe) {
    b = k.d - (j > k.m ? 1 : 0);
  } else if (P.layout == kBasic) {
    b = k.p - j * L;
  } else {
    const int c = L >> 1, second = (2 * P.D - 1 - j) * c;
    b = k.p >= second ? k.p - second + c : min(k.p - j * c, c - 1);
  }
  return max(-1, min(b, L - 1));
}

// The weights P of the backward kernels, up to the products with dS, are kept as halves (2^-11) times
// 2^kWeightShift, and the results multiplied by kWeightUnit: half numbers lose bits below 2^-14, so
// that without it a weight of 2^-18, one of 2^18 equal keys or of a key whose score lies 12 below the
// others', was off by 2^-8, and one of 2^-26 was 0. Now weights keep their 11 bits down to 2^-28 and
// are 0 below 2^-39. There is room for P up to 4, where rounding of an lse of millions would take it.
constexpr float kWeightShift = 14.f, kWeightUnit = 1.f / 16384.f;

// ---- query blocks: what the producer warp works out of an item ahead of the other warps, which
// would have to wait for the arithmetic (12000 cycles of a 60000-cycle item, measured) ----------
struct WinSeg {
  uint8_t j, sk;           // K/V shard, its sink rows (<= 128)
  uint16_t sink;           // its tiles (TileSet)
  int s0, n0, s1, n1;
};
__device__ __forceinline__ TileSet tiles_of(const WinSeg& g) { return {g.sink, g.s0, g.n0, g.s1, g.n1}; }
__device__ __forceinline__ WinSeg seg_of(int j, int sk, const TileSet& t) {
  return {static_cast<uint8_t>(j), static_cast<uint8_t>(sk), static_cast<uint16_t>(t.sink), t.s0, t.n0, t.s1, t.n1};
}
__device__ __forceinline__ bool has_tile(const TileSet& t, int b) {
  return (t.sink && b == 0) || (b >= t.s0 && b < t.s0 + t.n0) || (b >= t.s1 && b < t.s1 + t.n1);
}
struct WinSlot {
  int item;       // >= n_items: the end
  int tiles, nseg;
  int h, r, L, a0, a1;  // query head, rank, local length, first and last row of the block
  int row, lse;   // shard-major row of a0; element of lse of a0
  WinSeg seg[kMaxWindowShards];
};

// Fills in a slot for query rows a0 .. a1 of rank r (the whole warp): of one query tile, or with HALVES
// of two, whose own tiles go to half[2 * kMaxWindowShards], one after the other.
template <bool HALVES>
__device__ __forceinline__ void fill_slot(WinSlot& w, WinSeg* half, const Plan& P, int seq, int h, int r, int a0,
                                          int a1) {
  const SeqDesc& sd = P.seq[seq];
  const int lane = threadIdx.x & 31, L = sd.L, mid = HALVES ? min(a1 + 1, a0 + kQTileRows) : a1 + 1;
  int nseg = 0, tiles = 0;
  for (int base = 0; base < P.D; base += 32) {
    TileSet t = {0, 0, 0, 0, 0}, t0 = t, t1 = t;
    const int j = base + lane < P.D ? shard_at_step(P.D, r, base + lane) : 0;
    if (base + lane < P.D) {
      t = t0 = window_kv_tiles(P, L, r, j, a0, mid - 1);
      if (HALVES && mid <= a1) t = both_tiles(t0, t1 = window_kv_tiles(P, L, r, j, mid, a1));
    }
    const int n = tile_count(t);
    const unsigned some = __ballot_sync(0xffffffffu, n > 0);
    if (n > 0) {
      const int at = nseg + __popc(some & ((1u << lane) - 1u)), sk = sink_rows(P, L, j);
      w.seg[at] = seg_of(j, sk, t);
      if constexpr (HALVES) {
        half[at] = seg_of(j, sk, t0);
        half[kMaxWindowShards + at] = seg_of(j, sk, t1);
      }
    }
    nseg += __popc(some);
    tiles += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
  if (lane == 0) {
    w.tiles = tiles;
    w.nseg = nseg;
    w.h = h;
    w.r = r;
    w.L = L;
    w.a0 = a0;
    w.a1 = a1;
    w.row = sd.row_off + r * P.shard_stride + a0;
    w.lse = sd.lse_off + h * P.lse_hstride + r * P.shard_stride + a0;
  }
  __syncwarp();
}

}  // namespace ra
