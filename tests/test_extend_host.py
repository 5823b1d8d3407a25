"""Attention of several new tokens over a paged cache, on the CPU: which key tiles a block of rows
walks and how the walks are dealt out (csrc/ra_extend.h, the kernels' own arithmetic, compiled for the
host) against masks key by key; and the refusals of the calls, which come before any launch. The
pointers are never followed."""
import ctypes
import os
import subprocess

import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from context_blockwise_attention_step_gb300 import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "context_blockwise_attention_step_gb300", "csrc")
FAKE = 256

SOURCE = r"""
#include <algorithm>
#include <cstddef>
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "ra_extend.h"
using namespace ra;

static long blocks = 0, wrong = 0;
static void bad(const char* what, const ExtShape& s, const ExtSeg& g, int i) {
  if (wrong++ < 5)
    printf("%s: bt %d tile %d window %d sinks %d, n %d base %d k0 %d k1 %d shared %d, block %d\n", what, s.bt,
           1 << s.shift, s.window, s.sinks, g.n, g.base, g.k0, g.k1, g.shared, i);
}

int main() {
  srand(3);
  for (int it = 0; it < 30000; ++it) {
    ExtShape s;
    const int heads = 1 + rand() % 20, keys = rand() % 3 ? 128 : 64;
    s.shift = keys == 128 ? 7 : 6;
    s.half = keys / heads;
    s.wide = keys == 128 ? 2 : 1;
    s.lead = rand() % 3;
    s.bt = s.wide * s.half;
    s.window = rand() % 2 ? 1 + rand() % 1500 : 0;
    s.sinks = s.window && rand() % 3 ? rand() % 129 : 0;
    ExtSeg g = {};
    g.n = 1 + rand() % (rand() % 2 ? 10 : 900);
    g.base = rand() % (rand() % 2 ? 3000 : 50);
    if (!s.window && rand() % 2) g.k0 = g.base >> s.shift << s.shift;
    if (!s.window && rand() % 5 == 0) {
      g.shared = 1;
      g.k0 = 0;
      g.k1 = (1 + rand() % 50) << s.shift;
    }
    const int nb = ext_blocks(s, g.n);
    int64_t units = 0;
    for (int i = 0; i < nb; ++i, ++blocks) {
      if (ext_units_before(s, g, i) != units) bad("units before a block", s, g, i);
      const ExtWalk w = ext_walk(s, g, i);
      std::vector<char> seen((g.base + g.n + g.k1) / keys + 2, 0);  // the mask, key by key
      if (g.shared)
        for (int k = 0; k < g.k1; k += keys) seen[k / keys] = 1;
      else
        for (int j = i * s.bt; j < std::min(g.n, (i + 1) * s.bt); ++j)
          for (int p = g.base + j, k = g.k0; k <= p; ++k)
            if (!s.window || k > p - s.window || k < s.sinks) seen[k / keys] = 1;
      std::vector<int> want, got;
      for (size_t t = 0; t < seen.size(); ++t)
        if (seen[t]) want.push_back(static_cast<int>(t));
      for (int j = 0; j < w.count; ++j) got.push_back(ext_tile(w, j));
      if (got != want) bad("the tiles of a block", s, g, i);
      const int64_t all = s.lead + int64_t(w.count) * ext_weight(s, g, i);
      for (int64_t x : {int64_t(0), all - 1})
        if (ext_block_of(s, g, units + x) != i) bad("the block of a unit", s, g, i);
      units += all;
    }
    if (ext_units_before(s, g, nb) != units) bad("all units", s, g, nb);
  }
  // every tile belongs to one CTA, and the CTAs of a block's tiles behind its first are neighbours: none
  // between has no part
  for (int it = 0; it < 20000; ++it) {
    const ExtSeg seg = {};
    const int nb = 1 + rand() % 40;
    ExtShape s = {};
    s.wide = 1 + rand() % 2;
    s.lead = rand() % 12;
    s.least = s.wide + rand() % 8;
    std::vector<int> count, weight;
    int64_t units = 0;
    for (int i = 0; i < nb; ++i) {
      count.push_back(1 + rand() % 30);
      weight.push_back(s.wide == 2 && rand() % 2 ? 2 : 1);
      units += ext_units(s, count[i], weight[i]);
    }
    const int ctas = ext_ctas(s, units, 1 + rand() % 152);
    std::vector<std::vector<int>> owner(nb);
    for (int c = 0; c < ctas; ++c) {
      const int64_t u0 = ext_first(units, ctas, c), u1 = ext_first(units, ctas, c + 1);
      int64_t base = 0;
      for (int i = 0; i < nb; base += ext_units(s, count[i], weight[i]), ++i)
        for (int j = ext_tile_from(s, base, weight[i], count[i], u0); j < ext_tile_from(s, base, weight[i], count[i], u1);
             ++j) {
          owner[i].push_back(c);
          if (ext_cta_of(units, ctas, ext_tile_unit(s, base, weight[i], j)) != c) bad("the CTA of a tile", s, seg, i);
        }
    }
    for (int64_t i = 0, base = 0; i < nb; base += ext_units(s, count[i], weight[i]), ++i) {
      if (static_cast<int>(owner[i].size()) != count[i]) bad("tiles without a CTA", s, seg, i);
      for (size_t j = 1; j < owner[i].size(); ++j)
        if (owner[i][j] < owner[i][j - 1] || (j > 1 && owner[i][j] > owner[i][j - 1] + 1)) bad("a CTA without a part", s, seg, i);
      // the CTAs that the join looks for a block's parts at
      const ExtCtas of = ext_ctas_of(s, units, ctas, base, weight[i], count[i]);
      std::vector<int> at = {of.c0}, have = owner[i];
      for (int c = of.c0 + of.skip + 1; c <= of.c1; ++c) at.push_back(c);
      have.erase(std::unique(have.begin(), have.end()), have.end());
      if (at != have) bad("the CTAs of a block", s, seg, static_cast<int>(i));
    }
  }
  // far positions: in 64 bits
  {
    ExtShape s = {2, 1, 2, 1, 3, 7, 0, 0};
    ExtSeg g = {};
    g.n = 1000;
    g.base = 2147483584 - 1000;
    int64_t sum = 0;
    for (int i = 0; i < ext_blocks(s, g.n); ++i) sum += ext_units(s, ext_walk(s, g, i).count, ext_weight(s, g, i));
    if (sum != ext_units_before(s, g, ext_blocks(s, g.n))) bad("far positions", s, g, 0);
    s.window = 2147483647;
    if (sum != ext_units_before(s, g, ext_blocks(s, g.n))) bad("a window over everything", s, g, 0);
  }
  printf("%ld blocks checked, %ld wrong\n", blocks, wrong);
  return wrong != 0;
}
"""


@pytest.fixture(scope="module", autouse=True)
def built_library():
    ra.build()
    return _abi.lib()


def test_walks_and_shares(tmp_path):
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout
    assert int(res.stdout.split()[0]) > 100000


def _cache(**kw):
    c = _abi.RaPagedCache()
    base = dict(dtype=_abi.RA_BF16, hkv=2, head_dim=128, page_size=16, n_pages=8, n_seqs=3, max_pages=4,
                table_stride=4, page_stride=16 * 256, slot_stride=256, head_stride=128, k_pages=FAKE,
                v_pages=FAKE, block_table=FAKE)
    base.update(kw)
    for k, v in base.items():
        setattr(c, k, v)
    return c


def _extend(c=None, shared=None, n=5, hq=8, scale=0.0, window=0, sinks=0, q=FAKE, lens=FAKE, cu=FAKE, out=FAKE,
            lse=FAKE, ws=FAKE, size=1 << 40):
    c = _cache() if c is None else c
    s = None if shared is None else ctypes.byref(shared)
    return _abi.lib().ra_paged_attn_extend(ctypes.byref(c), s, n, hq, scale, window, sinks, q, lens, cu, out, lse, ws,
                                           size, None)


def test_refusals():
    bad, shape, unsupported = _abi.RA_ERR_INVALID_ARG, _abi.RA_ERR_SHAPE, _abi.RA_ERR_UNSUPPORTED
    for name in ("q", "lens", "out", "lse", "ws"):
        assert _extend(**{name: None}) == bad
    assert _extend(ws=128) == bad
    assert _extend(cu=None) == shape                     # 5 tokens of 3 sequences
    assert _extend(n=-1) == bad
    assert _extend(hq=7) == unsupported
    assert _extend(hq=0) == unsupported
    assert _extend(n=1 << 28) == unsupported             # 2^31 rows
    assert _extend(scale=float("nan")) == bad
    assert _extend(scale=float("inf")) == bad
    assert _extend(window=-1) == bad
    assert _extend(window=4, sinks=_abi.RA_MAX_SINKS + 1) == bad
    assert _extend(window=4, sinks=-1) == bad
    for kw in (dict(q=FAKE + 8), dict(out=FAKE + 8), dict(c=_cache(k_pages=FAKE + 8)), dict(c=_cache(slot_stride=260)),
               dict(c=_cache(head_stride=4)), dict(c=_cache(page_stride=16 * 256 + 4))):
        assert _extend(**kw) == bad
    need = _abi.lib().ra_paged_extend_workspace_bytes(ctypes.byref(_cache()), 0, 5, 8)
    assert need > 0
    assert _extend(size=need - 1) == _abi.RA_ERR_WORKSPACE

    two = _abi.RaSharedPrefix(2, FAKE, FAKE)
    assert _extend(shared=_abi.RaSharedPrefix(2, None, FAKE)) == bad
    assert _extend(shared=_abi.RaSharedPrefix(2, FAKE, None)) == bad
    assert _extend(shared=_abi.RaSharedPrefix(-1, FAKE, FAKE)) == bad
    assert _extend(shared=_abi.RaSharedPrefix(4, FAKE, FAKE)) == shape   # of 3 sequences
    assert _extend(shared=two, window=4) == unsupported
    more = _abi.lib().ra_paged_extend_workspace_bytes(ctypes.byref(_cache()), 2, 5, 8)
    assert more >= need + 2 * 5 * 8 * (128 + 2) * 4
    assert _extend(shared=two, size=more - 1) == _abi.RA_ERR_WORKSPACE


def test_nothing_to_do_is_no_error():
    need = _abi.lib().ra_paged_extend_workspace_bytes(ctypes.byref(_cache()), 0, 0, 8)
    assert _extend(n=0, q=None, out=None, lse=None, size=need) == _abi.RA_OK
    none = _cache(n_seqs=0, block_table=None)
    assert _extend(c=none, n=0, cu=None, q=None, lens=None, out=None, lse=None) == _abi.RA_OK


@pytest.mark.parametrize("kw", [dict(dtype=7), dict(hkv=0), dict(head_dim=96), dict(table_stride=3),
                                dict(n_seqs=_abi.RA_MAX_CACHE_SEQS + 1), dict(k_pages=None)], ids=str)
def test_bad_caches(kw):
    assert _extend(c=_cache(**kw)) < 0
    assert _abi.lib().ra_paged_extend_workspace_bytes(ctypes.byref(_cache(**kw)), 0, 5, 8) == 0


def test_shared_prefixes_are_checked_in_python():
    cu, lens = torch.tensor([0, 2], dtype=torch.int32), torch.tensor([5], dtype=torch.int32)
    with pytest.raises(ValueError):
        ra.SharedPrefix(cu, lens)  # not on a GPU
