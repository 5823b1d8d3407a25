"""Attention of several new tokens over a paged cache, and over prefixes that sequences share, on the
GPU against float64.

Tolerances, from the arithmetic. A score is a sum of dh products, off by at most dh * 2^-23 * sum |q k|
scale, below 2^-13 at these sizes (dh 128, |q k| scale summed below 2^3); the exponential and the
sums add less than 2^-16. So every weight is off by 2^-12 relative at most, and lse by 2^-12 absolute
(and its own rounding, 2^-22 relative). bf16 rounds the weights (2^-8 relative) and the result (2^-8):
|out - ref| <= (2^-8 + 2^-11) sum_k p_k |v_k| + 2^-8 |ref|, for f32 2^-11 sum_k p_k |v_k|.
"""
import numpy as np
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from context_blockwise_attention_step_gb300 import _abi
from oracle import heads as H

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
BIG = 260_000_000  # bytes: no small cache


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


def f64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    """Sequences in a paged cache. news, lens: new tokens and lengths with them; groups: list of
    (number of sequences, prefix length): their first tokens are equal, and in the same pages as far as
    these are whole. NaN wherever nobody may look: behind a sequence's end, in pages of nobody, and
    (with a window) in pages that no row sees. capacity: rows of the block table that make the cache this many
    bytes at most (a small one is read sequence by sequence in decoding steps)."""

    def __init__(self, seed, dtype, hq, hkv, dh, page, lens, news=None, groups=(), order="pshd", window=0, sinks=0,
                 scale=1.0, capacity=0):
        self.rng = rng = np.random.default_rng(seed)
        self.dtype, self.hq, self.hkv, self.dh, self.page = dtype, hq, hkv, dh, page
        self.lens, self.news = list(lens), [1] * len(lens) if news is None else list(news)
        self.window, self.sinks = window, sinks
        n_seqs = len(lens)
        width = max(1, max(-(-n // page) for n in lens)) + 1
        width = max(width, -(-capacity // (n_seqs * page * hkv * dh * 2 * (2 if dtype == BF16 else 4))) + 1)
        table = np.full((n_seqs, width), 1 << 30, np.int64)  # a bad page: entries that nobody may look at
        kv = [(self._randn(max(n, 1), hkv, dh), self._randn(max(n, 1), hkv, dh)) for n in lens]
        self.cu_groups, self.prefix_lens, at = [0], [], 0
        for m, p in groups:
            live = [b for b in range(at, at + m) if lens[b] >= p and self.news[b] > 0]
            for b in live[1:]:
                for i in (0, 1):
                    kv[b][i][:p] = kv[live[0]][i][:p]
            at += m
            self.cu_groups.append(at)
            self.prefix_lens.append(p)
        self.kv = kv
        pages, owner = [], {}
        at = 0
        for m, p in groups:
            live = [b for b in range(at, at + m) if lens[b] >= p and self.news[b] > 0]
            for i in range(p // page):
                for b in live:
                    owner[b, i] = owner.get((live[0], i), len(pages))
                    if owner[b, i] == len(pages):
                        pages.append((b, i))
            at += m
        for b, n in enumerate(lens):
            for i in range(-(-n // page)):
                lo = n - self.news[b] - window + 1
                if window and (i + 1) * page <= lo and i * page >= sinks:
                    continue  # a page that the window has left behind
                if (b, i) not in owner:
                    owner[b, i] = len(pages)
                    pages.append((b, i))
        n_pages = len(pages) + 2
        perm = rng.permutation(n_pages)
        shape = {"pshd": (n_pages, page, hkv, dh), "phsd": (n_pages, hkv, page, dh), "wide": (n_pages, page, hkv, 2, dh)}[order]
        store = [torch.full(shape, float("nan"), dtype=dtype) for _ in range(1 if order == "wide" else 2)]
        view = {"pshd": lambda: store, "phsd": lambda: [t.transpose(1, 2) for t in store],
                "wide": lambda: [store[0][:, :, :, 0], store[0][:, :, :, 1]]}[order]()
        for (b, i), at in owner.items():
            table[b, i] = perm[at]
            for dst, src in zip(view, kv[b]):
                part = torch.from_numpy(src[i * page:min(lens[b], (i + 1) * page)]).to(dtype)
                dst[perm[at], :part.shape[0]] = part
        store = [t.cuda() for t in store]
        self.pages = {"pshd": lambda: store, "phsd": lambda: [t.transpose(1, 2) for t in store],
                      "wide": lambda: [store[0][:, :, :, 0], store[0][:, :, :, 1]]}[order]()
        self.table = torch.from_numpy(table).int().cuda()
        self.cache = ra.make_cache(*self.pages, self.table)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32).cuda()
        self.cu = np.concatenate([[0], np.cumsum(self.news)])
        self.cu_new = torch.from_numpy(self.cu).int().cuda()
        self.q = torch.from_numpy(self._randn(int(self.cu[-1]), hq, dh) * scale).to(dtype).cuda()
        self.shared = ra.SharedPrefix(torch.tensor(self.cu_groups, dtype=torch.int32).cuda(),
                                      torch.tensor(self.prefix_lens, dtype=torch.int32).cuda()) if groups else None

    def _randn(self, *shape):
        x = torch.from_numpy(self.rng.standard_normal(shape)).to(self.dtype)
        return x.double().numpy()

    def reference(self, scale=None):
        """out, lse and sum p |v| of every row."""
        n = int(self.cu[-1])
        out, mag = np.zeros((n, self.hq, self.dh)), np.zeros((n, self.hq, self.dh))
        lse = np.full((n, self.hq), -np.inf)
        q = f64(self.q)
        for b, m in enumerate(self.lens):
            rows = slice(self.cu[b], self.cu[b + 1])
            if m < self.news[b] or m == 0:
                continue
            ok = H.seen(self.news[b], m, self.window, self.sinks)
            k, v = self.kv[b][0][:m], self.kv[b][1][:m]
            s = self.dh ** -0.5 if scale is None else scale
            out[rows], l = H.masked_fwd(q[rows], k, v, ok, s)
            mag[rows], _ = H.masked_fwd(q[rows], k, np.abs(v), ok, s)
            lse[rows] = l.T
        return out, lse, mag

    def run(self, **kw):
        kw = {"cu_new": self.cu_new, "shared": self.shared, "window": self.window, "sinks": self.sinks, **kw}
        return ra.paged_attn_extend(self.q, self.cache, self.seq_lens, **kw)

    def check(self, out, lse, ref=None, what=""):
        want, want_lse, mag = self.reference() if ref is None else ref
        half = 2.0 ** -8 if self.dtype == BF16 else 0.0
        got, got_lse = f64(out), f64(lse)
        bad = ~(np.abs(got - want) <= (half + 2.0 ** -11) * mag + half * np.abs(want))
        assert not bad.any(), f"{what} out: {bad.sum()} of {bad.size} off, rows {np.unique(np.argwhere(bad)[:, 0])[:9]}"
        assert np.array_equal(np.isinf(got_lse), np.isinf(want_lse)), f"{what} lse infinities"
        with np.errstate(invalid="ignore"):
            off = np.nan_to_num(np.abs(got_lse - want_lse) - 2.0 ** -22 * np.abs(want_lse))
        assert off.max(initial=0.0) <= 2.0 ** -12, f"{what} lse {off.max():.2e}"
        assert ra.check_device_status() == _abi.RA_OK, ra.last_error()


EXTEND = [
    # dtype, hq, hkv, dh, page, lens, news, window, sinks
    (BF16, 4, 1, 128, 64, [1], [1], 0, 0),
    (BF16, 32, 8, 128, 64, [300], [300], 0, 0),
    (BF16, 8, 2, 64, 16, [700, 3, 0, 129, 128], [5, 3, 0, 1, 128], 0, 0),
    (BF16, 8, 8, 128, 48, [257, 90], [257, 1], 0, 0),            # one head a K/V head: 256 tokens a block
    (BF16, 12, 4, 64, 7, [200, 77], [130, 44], 0, 0),            # three heads, pages of one key a box
    (BF16, 6, 1, 128, 1, [150], [90], 0, 0),                     # pages of one token
    (BF16, 48, 1, 64, 128, [300, 5], [7, 5], 0, 0),              # 48 heads a K/V head: two tokens a tile
    (BF16, 130, 1, 64, 32, [140], [3], 0, 0),                    # more heads than rows of a tile
    (BF16, 8, 1, 128, 256, [1000], [17], 0, 0),                  # pages of two tiles
    (BF16, 8, 2, 64, 16, [900, 30, 700], [100, 30, 3], 70, 0),
    (BF16, 8, 2, 64, 16, [900, 30, 700, 0], [100, 30, 300, 0], 200, 5),
    (BF16, 4, 1, 128, 64, [600], [600], 1, 128),
    (BF16, 4, 4, 64, 32, [1500], [700], 130, 100),
    (F32, 4, 2, 64, 16, [300, 3, 0, 65], [5, 3, 0, 65], 0, 0),
    (F32, 8, 1, 128, 48, [200, 90], [70, 1], 0, 0),
    (F32, 6, 2, 33, 7, [100], [40], 0, 0),
    (F32, 70, 1, 8, 16, [100], [3], 0, 0),
    (F32, 2, 1, 1, 5, [70], [70], 0, 0),
    (F32, 4, 2, 96, 16, [400, 30], [100, 30], 70, 3),
    (F32, 4, 2, 100, 16, [400], [200], 33, 128),
]


@pytest.mark.parametrize("case", EXTEND, ids=lambda c: f"{str(c[0])[6:]}_{c[1]}x{c[2]}_dh{c[3]}_p{c[4]}_n{len(c[5])}_w{c[7]}")
def test_extend(case):
    dt, hq, hkv, dh, page, lens, news, window, sinks = case
    b = Batch(1, dt, hq, hkv, dh, page, lens, news, window=window, sinks=sinks)
    ref = b.reference()
    out, lse = b.run()
    b.check(out, lse, ref)
    again = b.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])  # bit for bit


SHARED = [
    # dtype, hq, hkv, dh, page, groups, own lengths (0: idle), news
    (BF16, 32, 8, 128, 64, [(6, 1024)], [1, 5, 64, 130, 0, 2], None),
    (BF16, 8, 8, 64, 16, [(5, 700), (1, 300), (4, 900), (2, 0)], [3, 40, 1, 7, 9, 5, 1, 1, 200, 2, 33, 0], None),
    (BF16, 4, 1, 128, 48, [(40, 1000)], [1 + i % 7 for i in range(40)], None),   # 160 rows a K/V head: two tiles
    (BF16, 16, 1, 64, 64, [(33, 640)], [1 + i % 3 for i in range(33)], None),    # 528 rows: three blocks
    (BF16, 8, 2, 128, 64, [(4, 1300)], [50, 20, 3, 9], [50, 12, 3, 1]),          # questions after a document
    (BF16, 12, 4, 64, 32, [(3, 512), (3, 900)], [10, 30, 2, 9, 9, 9], [10, 1, 2, 0, 9, 4]),
    (BF16, 4, 4, 64, 64, [(3, 130)], [1, 1, 1], None),                           # too short to share
    (F32, 8, 2, 64, 16, [(5, 700), (3, 333)], [3, 40, 0, 7, 9, 5, 1, 1], None),
    (F32, 6, 1, 40, 7, [(4, 500)], [50, 20, 3, 9], [50, 12, 3, 1]),
    (F32, 16, 1, 128, 64, [(9, 600)], [2] * 9, None),
    # several tokens each behind a prefix long enough to be shared
    (BF16, 8, 2, 128, 64, [(6, 5000)], [50, 20, 3, 9, 60, 7], [50, 12, 3, 1, 40, 2]),
    (BF16, 12, 4, 64, 32, [(3, 1700), (4, 2600)], [10, 30, 2, 9, 9, 9, 100], [10, 1, 2, 0, 9, 4, 90]),
    (BF16, 4, 4, 64, 64, [(5, 6000)], [300, 257, 200, 9, 40], [300, 257, 100, 1, 40]),
    (F32, 6, 1, 40, 7, [(6, 2000)], [12, 20, 3, 9, 5, 1], [12, 3, 1, 2, 5, 1]),
    # more heads a K/V head than the kernel for few rows takes; more than rows of a tile
    (BF16, 48, 1, 64, 64, [(5, 3000)], [12, 1, 3, 9, 70], [12, 1, 3, 2, 66]),
    (BF16, 130, 1, 128, 32, [(4, 2500)], [2, 1, 3, 2], [2, 1, 3, 1]),
    (BF16, 34, 2, 64, 64, [(7, 1000)], [2, 1, 0, 3, 2, 5, 1], None),
]


@pytest.mark.parametrize("case", SHARED, ids=lambda c: f"{str(c[0])[6:]}_{c[1]}x{c[2]}_dh{c[3]}_g{len(c[5])}_n{len(c[6])}")
def test_shared_prefixes(case):
    dt, hq, hkv, dh, page, groups, own, news = case
    prefix = [p for m, p in groups for _ in range(m)]
    lens = [p + n if n else 0 for p, n in zip(prefix, own)]
    b = Batch(2, dt, hq, hkv, dh, page, lens, news, groups=groups, capacity=BIG)
    ref = b.reference()
    how = {} if news else {"cu_new": None}
    out, lse = b.run(**how)
    b.check(out, lse, ref)
    again = b.run(**how)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    b.check(*b.run(shared=None, **how), ref, "nothing shared")
    if not news:
        if all(own):  # (offsets give an idle sequence no row)
            b.check(*b.run(shared=None), ref, "one token each, by offsets")
        b.check(*ra.paged_attn_decode(b.q, b.cache, b.seq_lens, shared=b.shared), ref, "decode")
        small = Batch(2, dt, hq, hkv, dh, page, lens, news, groups=groups)
        b.check(*ra.paged_attn_decode(small.q, small.cache, small.seq_lens, shared=small.shared), ref, "a small cache")
