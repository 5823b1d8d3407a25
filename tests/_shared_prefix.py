"""Sequences in a paged cache behind prefixes that groups of them share, on the GPU, with the float64
definition of their attention: for the tests of shared prefixes."""
import numpy as np
import torch

import context_blockwise_attention_step_gb300 as ra

BF16, F32 = torch.bfloat16, torch.float32
BIG = 260_000_000  # bytes: decoding steps over smaller caches read every sequence apart
HIDDEN = 1 << 30   # a page that is not there


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Prefixed:
    """`lead` sequences of no group, then groups (sequences, prefix length), whose members have own[b]
    keys (the news[b] new ones among them; 0: idle) behind the prefix. NaN where nobody may look. With
    `hide` only the first member of a group with new tokens has the pages of the prefix's whole key tiles in its
    row of the block table: the others' are indexes outside the cache, which are recorded if they are followed."""

    def __init__(self, seed, dtype, hq, hkv, dh, page, groups, own, news=None, lead=0, order="pshd", hide=True, scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(dtype)  # noqa: E731
        self.dtype, self.hq, self.hkv, self.dh = dtype, hq, hkv, dh
        prefix = [0] * lead + [p for m, p in groups for _ in range(m)]
        group = [-1] * lead + [i for i, (m, _) in enumerate(groups) for _ in range(m)]
        n = len(own)
        assert n == len(prefix)
        self.news = [1] * n if news is None else list(news)
        self.lens = [p + x if x else 0 for p, x in zip(prefix, own)]
        common = [(rand(p, hkv, dh), rand(p, hkv, dh)) for _, p in groups]
        self.kv = []
        for b in range(n):
            parts = rand(own[b], hkv, dh), rand(own[b], hkv, dh)
            self.kv.append(parts if group[b] < 0 or not own[b]
                           else tuple(torch.cat([c, x]) for c, x in zip(common[group[b]], parts)))
        elem = 2 if dtype == BF16 else 4
        need = [-(-m // page) for m in self.lens]
        width = max(max(need), BIG // (n * page * hkv * dh * 2 * elem) + 1)
        table = np.full((n, width), HIDDEN, np.int64)
        at, pages_of = 0, []
        for _, p in groups:
            pages_of.append(range(at, at + p // page))
            at += p // page
        for b in range(n):
            if own[b]:
                same = pages_of[group[b]] if group[b] >= 0 else ()
                table[b, :len(same)] = same
                table[b, len(same):need[b]] = range(at, at + need[b] - len(same))
                at += need[b] - len(same)
        perm = np.random.default_rng(seed).permutation(at + 2)
        table[table < at] = perm[table[table < at]]
        shape = {"pshd": (at + 2, page, hkv, dh), "phsd": (at + 2, hkv, page, dh), "wide": (at + 2, page, hkv, 2, dh)}[order]
        store = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(1 if order == "wide" else 2)]
        self.pages = (store if order == "pshd" else [t.transpose(1, 2) for t in store] if order == "phsd"
                      else [store[0][:, :, :, 0], store[0][:, :, :, 1]])
        for b in range(n):
            pos = torch.arange(self.lens[b], device="cuda")
            where = torch.from_numpy(table[b]).cuda()[pos // page]
            for dst, src in zip(self.pages, self.kv[b]):
                dst[where, pos % page] = src[:self.lens[b]]
        if hide:
            tile = 128 if dtype == BF16 else 64
            for i in range(len(groups)):
                live = [b for b in range(n) if group[b] == i and own[b]]
                first = next((b for b in live if self.news[b]), None)
                for b in live:
                    if b != first:
                        table[b, :prefix[b] // tile * tile // page] = HIDDEN
        self.table = torch.from_numpy(table).int().cuda()
        self.cache = ra.make_cache(*self.pages, self.table)
        self.seq_lens = ints(self.lens)
        self.cu = np.concatenate([[0], np.cumsum(self.news)])
        self.cu_new = None if news is None else ints(self.cu)
        self.shared = ra.SharedPrefix(ints(np.cumsum([lead] + [m for m, _ in groups])), ints([p for _, p in groups]))
        self.q = (torch.randn(int(self.cu[-1]), hq, dh, generator=g, device="cuda") * scale).to(dtype)

    def run(self, **kw):
        kw = {"cu_new": self.cu_new, "shared": self.shared, **kw}
        return ra.paged_attn_extend(kw.pop("q", self.q), kw.pop("cache", self.cache), kw.pop("seq_lens", self.seq_lens), **kw)

    def reference(self):
        """out and lse of every row, float64."""
        grp = self.hq // self.hkv
        out, lse = torch.zeros(self.q.shape, dtype=torch.float64, device="cuda"), None
        lse = torch.full(self.q.shape[:2], -float("inf"), dtype=torch.float64, device="cuda")
        for b, m in enumerate(self.lens):
            n, rows = self.news[b], slice(int(self.cu[b]), int(self.cu[b + 1]))
            if m == 0 or n == 0:
                continue
            k, v = (x.double() for x in self.kv[b])
            q = self.q[rows].double().view(n, self.hkv, grp, self.dh)
            s = torch.einsum("rhgd,khd->rhgk", q, k) * self.dh ** -0.5
            ahead = torch.arange(m, device="cuda") > torch.arange(m - n, m, device="cuda")[:, None]
            s = s.masked_fill(ahead[:, None, None], -float("inf"))
            out[rows] = torch.einsum("rhgk,khd->rhgd", torch.softmax(s, -1), v).reshape(n, self.hq, self.dh)
            lse[rows] = torch.logsumexp(s, -1).reshape(n, self.hq)
        return out, lse
