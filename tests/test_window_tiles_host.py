"""The K/V tiles that the windowed kernels walk, on the CPU: the kernels' own arithmetic
(csrc/ra_plan.h) compiled for the host, over every layout, odd shard lengths and windows below the
number of shards.

The forward walks the tiles of a block of two query tiles and hands each to the query tiles that see
it. A tile that neither sees is never released, so the block's tiles have to be the union of the two
query tiles' own; and a query tile's own have to hold every key that one of its rows sees.
"""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "context_blockwise_attention_step_gb300", "csrc")

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include <algorithm>
using std::min; using std::max;
#include "ra_plan.h"
using namespace ra;

static long checked = 0, wrong = 0;
static void bad(const char* what, const Plan& P, int L, int r, int j, int a0) {
  if (wrong++ < 5)
    printf("%s: layout %d D %d L %d window %d sinks %d rank %d shard %d row %d\n", what, P.layout, P.D, L, P.window,
           P.sinks, r, j, a0);
}
static std::vector<int> tiles(const TileSet& t) {
  std::vector<int> v;
  for (int i = 0; i < tile_count(t); ++i) v.push_back(tile_at(t, i));
  return v;
}

int main() {
  static Plan P;
  P.causal = 1;
  const int Ds[] = {1, 2, 3, 5, 8, 40, 64}, Ws[] = {1, 2, 3, 4, 7, 20, 63, 64, 127, 128, 129, 300, 1000};
  const int Ls[] = {1, 2, 126, 127, 128, 129, 130, 255, 256, 257, 258, 384, 385, 386, 513, 641}, Ss[] = {0, 1, 5, 128};
  for (int layout = 0; layout < 3; ++layout)
    for (int D : Ds) for (int L : Ls) for (int W : Ws) for (int S : Ss) {
      if (layout == kZigzag && L % 2) continue;
      if (D > 8 && (S == 5 || W == 300 || W == 7)) continue;  // (time)
      P.layout = layout; P.D = D; P.window = W; P.sinks = S;
      const int nt = ceil_div(L, kKvTileRows);
      for (int r = 0; r < D; ++r) for (int j = 0; j < D; ++j) for (int a0 = 0; a0 < L; a0 += kFwdBlockRows) {
        const int a1 = min(L, a0 + kFwdBlockRows) - 1, mid = min(a1 + 1, a0 + kQTileRows);
        TileSet h[2] = {window_kv_tiles(P, L, r, j, a0, mid - 1), {0, 0, 0, 0, 0}};
        if (mid <= a1) h[1] = window_kv_tiles(P, L, r, j, mid, a1);
        const std::vector<int> u = tiles(both_tiles(h[0], h[1]));
        std::vector<int> want;
        for (int t = 0; t < 2; ++t) for (int b : tiles(h[t])) want.push_back(b);
        std::sort(want.begin(), want.end());
        want.erase(std::unique(want.begin(), want.end()), want.end());
        ++checked;
        if (u != want) bad("the block's tiles are not the query tiles'", P, L, r, j, a0);
        for (int t = 0; t < 2; ++t) {
          const std::vector<int> v = tiles(h[t]);
          if (!std::is_sorted(v.begin(), v.end()) || std::adjacent_find(v.begin(), v.end()) != v.end() ||
              (!v.empty() && (v.front() < 0 || v.back() >= nt)))
            bad("a query tile's tiles are out of order or range", P, L, r, j, a0);
        }
        if (D > 8 || L > 400) continue;
        std::vector<char> in[2] = {std::vector<char>(nt), std::vector<char>(nt)};
        for (int t = 0; t < 2; ++t) for (int b : tiles(h[t])) in[t][b] = 1;
        for (int a = a0; a <= a1; ++a) {
          const int64_t p = layout_pos(layout, D, L, r, a);
          for (int k = 0; k < L; ++k) {  // the mask, key by key
            const int64_t x = layout_pos(layout, D, L, j, k);
            if (x > p) break;  // (positions grow with k)
            if ((x > p - W || x < S) && !in[a >= mid][k / kKvTileRows]) {
              bad("a visible key's tile is missing", P, L, r, j, a);
              break;
            }
          }
        }
      }
    }
  printf("%ld blocks checked, %ld wrong\n", checked, wrong);
  return wrong != 0;
}
"""


def test_a_block_walks_the_union_of_its_query_tiles(tmp_path):
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout
    assert int(res.stdout.split()[0]) > 100000


@pytest.mark.parametrize("D,L,window", [(2, 129, 1), (4, 129, 3), (3, 129, 2), (2, 385, 1), (8, 641, 5)])
def test_the_shapes_whose_block_has_a_key_between_its_query_tiles(D, L, window):
    """In the stripe layout the last row of a shard of 256 n + 129 rows is a query tile of its own;
    the key before it in an earlier shard lies outside its window, and inside no other row's."""
    r, j = D - 1, 0
    last = L - 1
    assert last % 256 == 128
    key = last * D + j           # the shard's last key, the first of its tile
    assert last % 128 == 0
    assert not any(p - window < key <= p for p in range(r, L * D, D))  # no row of rank r sees it
