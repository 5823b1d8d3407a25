// ra_extend.h — integer part of the attention of several new tokens over a paged cache: which keys
// a block of query rows walks, and how the walks are dealt out. Host and device.
//
// The work is a list of segments, each a run of query tokens against a run of keys:
//   prefix segment  the tokens of all sequences of a group against the keys [0, k1) that they
//                   share; every row sees every key
//   own segment     the tokens of one sequence, at positions base .. base + n - 1, against the
//                   keys [k0, base + n); row j sees the keys up to base + j, with a window only
//                   the last `window` of these and the first `sinks`
// k0 and k1 are whole key tiles. A segment's tokens are cut into blocks of `bt`; a block walks the
// key tiles that one of its rows sees. A tile of a block costs a unit if the block has at most
// `half` tokens, else `wide` units, a block `lead` units more (its start and end, counted with its first
// tile), and every CTA gets the same share of all units, in the order segment, pair (K/V head and
// block of its query heads), block, tile. A tile belongs to the CTA that its first unit falls to; with
// shares of `least` >= `wide` units, each CTA between that of a block's second tile and its last one's
// has a tile of it. (Between the first tile's and the second's there can be some whose share is all lead.)
//
// Segments are of two classes, each with a kernel, a shape and shares of its own: those of few rows
// (at most 16 a K/V head, all in one block), and the others.
#pragma once
#include <stdint.h>

#include "ra_layout.h"

namespace ra {

enum : int { kExtMany = 0, kExtFew = 1 };
constexpr int kExtFewRows = 16;  // a K/V head
RA_HD bool ext_few(int n, int group) { return n * static_cast<int64_t>(group) <= kExtFewRows; }

struct ExtShape {
  int32_t bt, half;  // tokens of a block, and of one that costs one unit a tile
  int32_t wide;      // units of a tile of a larger block: 1 or 2
  int32_t lead;      // units of a block beside its tiles'
  int32_t least;     // units of a CTA's share at least: `wide` or more
  int32_t shift;     // log2 of a tile's keys
  int32_t window, sinks;
};

struct ExtSeg {
  int64_t unit0[2];  // units of each class before this segment
  int64_t units;     // units of one pair, of the segment's class; 0: nothing to walk
  int32_t t0, n;   // first token row, tokens
  int32_t base;    // own: position of token t0
  int32_t k0, k1;  // own: first key, keys; prefix: 0, keys
  int32_t seq;     // row of the block table
  int32_t blocks0; // own blocks before this segment
  int32_t prefix;  // own: the prefix segment that has the keys before k0, or -1
  int32_t shared;  // a prefix segment: 1, or 2 where at least half of its rows are of sequences with few rows
  int32_t cls;
};

RA_HD int64_t ext_unit0(const ExtSeg& g, int cls) { return cls == kExtMany ? g.unit0[kExtMany] : g.unit0[kExtFew]; }

// a / b. (In 32 bits where they do: a division of 64 takes a hundred instructions.)
RA_HD int64_t ext_div(int64_t a, int64_t b) {
  return (a | b) >> 31 == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// Where the share of a CTA begins, and the block that its first unit falls to.
struct ExtStart {
  int64_t u0, base;  // base: the block's first unit (u1 is the next CTA's u0)
  int32_t seg, hk, hblk, blk;
};

// Tiles of a block: walk index j is tile j for j < ns (first tokens before the window), else
// first + j - ns.
struct ExtWalk {
  int32_t first, ns, count;
};
RA_HD int ext_tile(const ExtWalk& w, int j) { return j < w.ns ? j : w.first + j - w.ns; }

RA_HD int ext_blocks(const ExtShape& s, int n) { return n > 0 ? (n - 1) / s.bt + 1 : 0; }

// The lowest key of the window of block i's first row.
RA_HD int64_t ext_low(const ExtShape& s, const ExtSeg& g, int64_t i) {
  const int64_t at = g.base + i * s.bt - s.window + 1;
  return s.window > 0 && at > g.k0 ? at : g.k0;
}

RA_HD ExtWalk ext_walk(const ExtShape& s, const ExtSeg& g, int i) {
  const int kt = 1 << s.shift;
  if (g.shared) return {0, 0, (g.k1 + kt - 1) >> s.shift};
  const int64_t end = static_cast<int64_t>(i + 1) * s.bt;
  const int hi = g.base + static_cast<int>(end < g.n ? end : g.n);
  ExtWalk w;
  w.first = static_cast<int>(ext_low(s, g, i) >> s.shift);
  w.ns = 0;
  if (s.window > 0 && s.sinks > 0) {
    w.ns = (s.sinks + kt - 1) >> s.shift;
    if (w.ns > w.first) w.ns = w.first;
  }
  w.count = ((hi - 1) >> s.shift) - w.first + 1 + w.ns;
  return w;
}

// sum over i < n of floor((a i + b) / 2^shift); a >= 1, b >= 0: take out the whole parts, then count the
// lattice points below the line by the other axis, as Euclid's algorithm would go on (the reciprocity of
// such sums: Graham, Knuth, Patashnik, Concrete Mathematics, section 3.5)
RA_HD int64_t ext_floor_sum(int64_t n, int shift, int64_t a, int64_t b) {
  int64_t m = int64_t(1) << shift, sum = 0;
  while (n > 0) {
    if (a >= m) {
      sum += (n - 1) * n / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      sum += n * (b / m);
      b %= m;
    }
    const int64_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const int64_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

// Tiles of the blocks before block i <= blocks, all of them whole (i == blocks: the last one counted
// as whole, which it need not be).
RA_HD int64_t ext_tiles_before(const ExtShape& s, const ExtSeg& g, int64_t i) {
  const int64_t kt = int64_t(1) << s.shift;
  if (g.shared) return i * ((g.k1 + kt - 1) >> s.shift);
  int64_t sum = ext_floor_sum(i, s.shift, s.bt, g.base + kt + s.bt - 1);  // ends: (hi - 1) / kt + 1
  if (s.window <= 0) return sum - i * (g.k0 >> s.shift);
  const int64_t low = static_cast<int64_t>(g.base) - s.window + 1;  // of block 0; k0 is 0
  const int64_t skip = low >= 0 ? 0 : (-low + s.bt - 1) / s.bt;  // blocks whose window begins at key 0
  if (i > skip) sum -= ext_floor_sum(i - skip, s.shift, s.bt, low + skip * s.bt);
  if (s.sinks > 0) {
    const int64_t most = (s.sinks + kt - 1) >> s.shift;
    for (int64_t k = 1; k <= most; ++k) {  // blocks whose window begins at tile k or later
      const int64_t need = k * kt - low, from = need <= 0 ? 0 : (need + s.bt - 1) / s.bt;
      if (i > from) sum += i - from;
    }
  }
  return sum;
}

// Units of a tile of block i, of the block, and of the blocks before block i <= blocks (of one pair).
RA_HD int ext_weight(const ExtShape& s, const ExtSeg& g, int i) {
  return g.n - static_cast<int64_t>(i) * s.bt > s.half ? s.wide : 1;
}
RA_HD int64_t ext_units(const ExtShape& s, int count, int weight) { return s.lead + static_cast<int64_t>(count) * weight; }
RA_HD int64_t ext_units_before(const ExtShape& s, const ExtSeg& g, int i) {
  const int nb = ext_blocks(s, g.n);
  if (i <= 0 || nb == 0) return 0;
  const int whole = i < nb ? i : nb - 1;  // blocks that are certainly whole
  const int64_t units = whole == 0 ? 0 : ext_tiles_before(s, g, whole) * s.wide + static_cast<int64_t>(whole) * s.lead;
  return i < nb ? units : units + ext_units(s, ext_walk(s, g, nb - 1).count, ext_weight(s, g, nb - 1));
}
// The block that unit u of a pair falls to.
RA_HD int ext_block_among(const ExtShape& s, const ExtSeg& g, int64_t u) {
  int lo = 0, hi = ext_blocks(s, g.n) - 1;
  if (g.shared) {  // all blocks alike but the last
    const int64_t i = ext_div(u, ext_units(s, ext_walk(s, g, 0).count, s.wide));
    return i < hi ? static_cast<int>(i) : hi;
  }
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (ext_units_before(s, g, mid) <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}
RA_HD int ext_block_of(const ExtShape& s, const ExtSeg& g, int64_t u) {
  return g.n <= s.bt ? 0 : ext_block_among(s, g, u);
}

// Shares: of `units` units CTA i of `ctas` has [ext_first(i), ext_first(i + 1)).
RA_HD int ext_ctas(const ExtShape& s, int64_t units, int most) {
  if (units >= static_cast<int64_t>(most) * s.least) return most;
  const int64_t c = units / s.least;
  return static_cast<int>(c < 1 ? (units > 0 ? 1 : 0) : c);
}
RA_HD int64_t ext_first(int64_t units, int ctas, int i) { return ext_div(units * i, ctas); }
RA_HD int ext_cta_of(int64_t units, int ctas, int64_t u) {
  return static_cast<int>(ext_div((u + 1) * ctas - 1, units));
}
// The first unit of tile j of a block (its own first unit is `base`), and the first tile of a block of
// `count` tiles of `weight` units whose first unit is not before unit u.
RA_HD int64_t ext_tile_unit(const ExtShape& s, int64_t base, int weight, int j) {
  return j == 0 ? base : base + s.lead + static_cast<int64_t>(j) * weight;
}
RA_HD int ext_tile_from(const ExtShape& s, int64_t base, int weight, int count, int64_t u) {
  if (u <= base) return 0;
  const int64_t past = u - base - s.lead;
  const int64_t j = past <= weight ? 1 : (past + weight - 1) >> (weight - 1);  // weight is 1 or 2
  return j < count ? static_cast<int>(j) : count;
}

// The CTAs that have tiles of a block: c0, and c0 + skip + 1 .. c1.
struct ExtCtas {
  int32_t c0, skip, c1;
};
RA_HD ExtCtas ext_ctas_of(const ExtShape& s, int64_t units, int ctas, int64_t base, int weight, int count) {
  ExtCtas c;
  c.c0 = ext_cta_of(units, ctas, base);
  c.c1 = ext_cta_of(units, ctas, ext_tile_unit(s, base, weight, count - 1));
  const int second = count < 2 ? c.c0 : ext_cta_of(units, ctas, ext_tile_unit(s, base, weight, 1));
  c.skip = second > c.c0 ? second - c.c0 - 1 : 0;
  return c;
}

// The units that a tile of a prefix costs the blocks of n tokens, and whether to share a prefix of `tiles`
// tiles that cost a group's sequences, each by itself, `apart` units a tile, and all together `together`.
// Sharing leaves two float parts of every row in memory, written and read once, and makes two blocks of
// one: it has to save a dozen tiles of the row's block. (us shared and apart, bf16, behind the tiles that
// each of the blocks together saves: 32/8 heads of 128, 16 questions of up to 100 tokens behind 4096 keys, 9.9: 117 and 108; of 300 behind 16384,
// 10: 661 and 615; 8 of 40 behind 16384, 107: 84 and 154. 8/8 heads of 64, 4 of 1000 behind 16384, 8.5: 209
// and 209; 16 of 500, 21: 252 and 258; 8 of 40 behind 1024, 24: 37 and 40; 16 of 300, 39: 186 and 236.)
RA_HD int64_t ext_block_units(const ExtShape& s, int64_t n) {
  if (n <= 0) return 0;
  const int64_t nb = (n - 1) / s.bt + 1;
  return (nb - 1) * s.wide + (n - (nb - 1) * s.bt > s.half ? s.wide : 1);
}
RA_HD bool ext_worth_sharing(int64_t tiles, int64_t apart, int64_t together) {
  return tiles > 0 && tiles * (apart - together) > 12 * together;
}

}  // namespace ra
