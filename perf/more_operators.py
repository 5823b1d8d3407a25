"""Timed cases of the operators for models whose tokens have positions on several axes, and for
batches that go on from a common prefix:

  norm_axes    the queries and keys of a training step in shard-major order: per-head
               root-mean-square norm and a rotation whose pairs turn by the token's position on
               one of several axes (time, height, width), forward and backward
  append_axes  new tokens of running sequences into the pages of a cache, q and k normed and
               rotated in the same way
  shared       attention of one new token of every sequence over a paged cache in which groups of
               sequences begin with the same prefix
  extend       causal attention of several new tokens of every sequence over the paged cache that
               holds them already, with or without a common prefix, or through a window

``run`` computes a case in elementary torch operations (float32, angles in float64) or, with
``own`` set, by the framework's calls. ``exact`` is the definition in float64.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
BASE = 500000.0


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # a short training batch of text and images: many small heads, where launches count
        dict(name="norm_axes_b2_s4096_h8_dh64", op="norm_axes", dtype="bf16", layout="basic", D=4,
             hq=8, hkv=8, dh=64, batch=2, seqlen=4096, n_seqs=0, rotary=64, interleaved=False,
             sections="8,12,12", cyclic=False, ladder="one"),
        # one long context of text and video of a grouped-query model, the axes taken in turn
        dict(name="norm_axes_s131072_gqa32x8_dh128", op="norm_axes", dtype="bf16", layout="zigzag",
             D=16, hq=32, hkv=8, dh=128, batch=1, seqlen=131072, n_seqs=0, rotary=128,
             interleaved=False, sections="24,20,20", cyclic=True, ladder="one"),
        # the float32 path: packed images with a row and a column, each with frequencies of its own
        dict(name="norm_axes_f32_varlen_dh96", op="norm_axes", dtype="f32", layout="stripe", D=8,
             hq=4, hkv=2, dh=96, batch=0, seqlen=8192, n_seqs=5, rotary=48, interleaved=True,
             sections="12,12", cyclic=False, ladder="own"),
        # one decoding step of a small batch: latency
        dict(name="append_axes_b4_decode", op="append_axes", dtype="bf16", hq=32, hkv=8, dh=128,
             batch=4, new_max=1, old_max=4096, page=64, rotary=128, interleaved=False,
             sections="16,24,24", cyclic=False, ladder="one"),
        # prompts of sixteen sequences with images in them that go into the cache at once
        dict(name="append_axes_16_prompts_s8192", op="append_axes", dtype="bf16", hq=32, hkv=8,
             dh=128, batch=16, new_max=8192, old_max=100, page=64, rotary=128, interleaved=False,
             sections="16,24,24", cyclic=False, ladder="one"),
        # a few answers sampled from one short prompt: latency
        dict(name="shared_b8_prefix960", op="shared", dtype="bf16", hq=32, hkv=8, dh=128, batch=8,
             groups=1, prefix=960, own_max=40, page=64),
        # many questions about one long document
        dict(name="shared_b64_prefix32768", op="shared", dtype="bf16", hq=32, hkv=8, dh=128,
             batch=64, groups=1, prefix=32768, own_max=500, page=64),
        # requests of six programs, each with instructions of its own, some sequences alone or idle
        dict(name="shared_b96_6_prefixes_dh64", op="shared", dtype="bf16", hq=8, hkv=8, dh=64,
             batch=96, groups=6, prefix=10000, own_max=700, page=16),
        # the float32 path
        dict(name="shared_f32_b16_prefix4096", op="shared", dtype="f32", hq=16, hkv=4, dh=64,
             batch=16, groups=1, prefix=4096, own_max=300, page=64),
        # four drafted tokens of every sequence of a model with a window, to be checked in one pass
        dict(name="extend_b33_draft4_window1024_dh64", op="extend", dtype="bf16", hq=8, hkv=8,
             dh=64, batch=33, groups=0, prefix=0, new_max=4, max_len=16384, page=16, window=1024,
             sinks=4),
        # sixteen questions of up to 500 tokens after one long document
        dict(name="extend_16_questions_prefix16384", op="extend", dtype="bf16", hq=32, hkv=8,
             dh=128, batch=16, groups=1, prefix=16384, new_max=500, max_len=16884, page=64,
             window=0, sinks=0),
        # a long prompt that comes in chunks: the last one, after all the others
        dict(name="extend_chunk4096_s32768", op="extend", dtype="bf16", hq=32, hkv=8, dh=128,
             batch=1, groups=0, prefix=0, new_max=4096, max_len=32768, page=64, window=0, sinks=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_axes", "append_axes", "shared", "shared", "extend", "extend"])
    hq, hkv = rng.choice([(8, 8), (4, 2), (16, 16), (32, 8), (8, 1), (12, 4), (6, 2)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dh = rng.choice([64, 128]) if dtype == "bf16" else rng.choice([32, 48, 64, 96, 128])
    c = dict(op=op, dtype=dtype, hq=hq, hkv=hkv, dh=dh)
    page = rng.choice([16, 64, 128, 48])
    if op in ("norm_axes", "append_axes"):
        rotary = rng.choice([dh, dh // 2])
        n_axes = rng.choice([2, 3, 3])
        last = rotary // 2 // n_axes + rng.choice([0, 1])
        sections = [rotary // 2 - (n_axes - 1) * last] + [last] * (n_axes - 1)
        c.update(rotary=rotary, interleaved=rng.random() < 0.3,
                 sections=",".join(str(x) for x in sections), cyclic=rng.random() < 0.4,
                 ladder=rng.choice(["one", "own"]))
        if op == "append_axes":
            one = rng.random() < 0.5
            return dict(c, page=page, batch=_log_int(rng, 1, 200) if one else rng.choice([1, 3, 16]),
                        new_max=1 if one else _log_int(rng, 2, 2900), old_max=_log_int(rng, 1, 500))
        D, n_seqs = rng.choice([1, 2, 3, 4, 8]), rng.choice([0, 0, 3, 7, 16])
        batch = 0 if n_seqs else rng.choice([1, 2, 3])
        unit = 2 * D * max(1, batch)
        n = max(unit, _log_int(rng, 64, 65536 if dtype == "bf16" else 8192) // unit * unit)
        return dict(c, layout=rng.choice(["basic", "zigzag", "stripe"]), D=D, batch=batch,
                    seqlen=n // max(1, batch), n_seqs=n_seqs)
    if op == "shared":
        batch = _log_int(rng, 2, 128)
        groups = rng.choice([1, 1, 2, 5]) if batch >= 10 else 1
        most = (32768 if dtype == "bf16" else 4096) // groups
        return dict(c, batch=batch, groups=groups, prefix=_log_int(rng, 1, most),
                    own_max=_log_int(rng, 1, 700), page=page)
    batch, new = rng.choice([1, 1, 3, 16, 33]), _log_int(rng, 1, 1000)
    groups = 1 if batch > 1 and rng.random() < 0.5 else 0
    most = max(new, min(32768, (1 << (30 if dtype == "bf16" else 27)) // (batch * new * hq)))
    prefix = _log_int(rng, 1, max(1, most - new)) if groups else 0
    max_len = prefix + new + _log_int(rng, 1, 100) if groups else max(new, _log_int(rng, 1, most))
    w = not groups and rng.random() < 0.4
    return dict(c, batch=batch, groups=groups, prefix=prefix, new_max=new, max_len=max_len,
                page=page, window=_log_int(rng, 1, max_len) if w else 0,
                sinks=rng.choice([0, 1, 4, 16]) if w else 0)


# ------------------------------------------------------------------------------ shapes

def _lengths(case):
    """Natural-order lengths of a training case: copies of seqlen, or a fixed uneven split of
    seqlen tokens into n_seqs pieces that the layout divides."""
    if case["batch"] > 0:
        return [case["seqlen"]] * case["batch"]
    unit, n = 2 * case["D"], case["n_seqs"]
    total = case["seqlen"] // unit
    weights = [1.0 + (i * 7 % 11) for i in range(n)]
    out = [int(total * w / sum(weights)) for w in weights]
    out[-1] += total - sum(out)
    return [x * unit for x in out]


def _natural_rows(case):
    """The natural row of every shard-major row."""
    lens, D, layout = _lengths(case), case["D"], case["layout"]
    starts = np.concatenate([[0], np.cumsum(lens)])
    pieces = {}
    for i, n in enumerate(lens):
        L = n // D
        for r in range(D):
            a = np.arange(L)
            if layout == "basic":
                pos = r * L + a
            elif layout == "stripe":
                pos = a * D + r
            else:
                c = L // 2
                pos = np.where(a < c, r * c + a, (2 * D - 1 - r) * c + a - c)
            pieces[i, r] = starts[i] + pos
    order = ([(i, r) for i in range(len(lens)) for r in range(D)] if case["batch"] > 0
             else [(i, r) for r in range(D) for i in range(len(lens))])
    return np.concatenate([pieces[k] for k in order]).astype(np.int64)


def _axis_positions(n, n_axes, rng):
    """Positions of n tokens. Two axes: rows and columns of one image. Three: text, whose tokens
    have one position on every axis, and videos, whose patches have a frame, a row and a column
    from the text before them on."""
    out = np.zeros((n, n_axes), dtype=np.int32)
    if n_axes == 2:
        width = int(rng.integers(20, 100))
        out[:, 0], out[:, 1] = np.arange(n) // width, np.arange(n) % width
        return out
    at, p = 0, 0
    while at < n:
        m = min(n - at, int(rng.integers(1, 300)))
        out[at:at + m] = (p + np.arange(m))[:, None]
        at, p = at + m, p + m
        t, h, w = (int(rng.integers(1, top)) for top in (9, 33, 33))
        m = min(n - at, t * h * w)
        i = np.arange(m)
        out[at:at + m] = p + np.stack([i // (h * w), i // w % h, i % w], -1)
        at, p = at + m, p + max(t, h, w)
    return out


def _axis_of(case):
    """The axis of every rotated pair: runs of the sections' lengths, or (cyclic) in turn for as
    long as a section lasts, and the first axis for the rest."""
    sections = [int(x) for x in case["sections"].split(",")]
    n = len(sections)
    if not case["cyclic"]:
        return [a for a, s in enumerate(sections) for _ in range(s)]
    return [i % n if i < n * sections[i % n] else 0 for i in range(sum(sections))]


def _frequencies(case):
    """Radians per position of every pair: one ladder over all pairs, or one for each axis."""
    half = case["rotary"] // 2
    if case["ladder"] == "one":
        return [BASE ** (-i / half) for i in range(half)]
    axis = _axis_of(case)
    seen, out = {}, []
    for a in axis:
        seen[a] = seen.get(a, -1) + 1
        out.append(10000.0 ** (-seen[a] / axis.count(a)))
    return out


def _rolled(x, seed):
    """The same numbers for every seed, in another order."""
    k = seed % len(x) if len(x) else 0
    return x[k:] + x[:k]


def _append_lengths(case, seed):
    """New tokens of each sequence, and its tokens in the cache before them."""
    b, hi = case["batch"], case["new_max"]
    new = [max(1, hi - i * (hi - 1) // max(1, b - 1)) for i in range(b)]
    old = [i * 37 % (case["old_max"] + 1) for i in range(b)]
    return new, _rolled(old, seed)


def _shared_lengths(case, seed):
    """Group starts, prefix lengths (whole pages, but for one shorter than a page), and each
    sequence's own tokens; from five sequences on one sequence is idle (-1)."""
    b, g, page = case["batch"], case["groups"], case["page"]
    starts = [0] + sorted({max(1, min(b, round(b * ((i + 1) / g) ** 1.3))) for i in range(g)})
    prefixes = []
    for i in range(len(starts) - 1):
        p = max(1, case["prefix"] * (len(starts) - 1 - i) // (len(starts) - 1))
        prefixes.append(p // page * page if p >= page else p)
    mine = _rolled([1 + i * 53 % case["own_max"] for i in range(b)], seed)
    if b >= 5:
        mine[seed % b] = -1
    return starts, prefixes, mine


def _extend_lengths(case, seed):
    """New tokens of each sequence and its length with them."""
    b, hi = case["batch"], case["new_max"]
    new = _rolled([max(1, hi - i * 29 % hi) for i in range(b)], seed)
    if case["groups"]:
        lens = [case["prefix"] + n + (i * 17 % max(1, case["max_len"] - case["prefix"] - hi + 1))
                for i, n in enumerate(new)]
    else:
        lens = [max(n, case["max_len"] - i * (case["max_len"] // (b + 1))) for i, n in enumerate(new)]
    return new, lens


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, dh = case["hq"], case["hkv"], case["dh"]
    if case["op"] == "norm_axes":
        rows = sum(_lengths(case))
        n = rows * (hq + hkv) * dh
        return {"bytes": 5 * n * es + 2 * dh * es + 2 * dh * 4 + 2 * rows * 4 * len(case["sections"].split(",")),
                "flops": 30 * n}
    if case["op"] == "append_axes":
        rows = sum(_append_lengths(case, 1)[0])
        return {"bytes": 2 * rows * (hq + 2 * hkv) * dh * es + 8 * case["batch"] +
                rows * 4 * len(case["sections"].split(",")),
                "flops": 10 * rows * (hq + hkv) * dh}
    if case["op"] == "shared":
        starts, prefixes, mine = _shared_lengths(case, 1)
        rows, keys, pairs = case["batch"], 0, 0
        for i, p in enumerate(prefixes):
            live = [n for n in mine[starts[i]:starts[i + 1]] if n >= 0]
            keys += p * bool(live) + sum(live)
            pairs += sum(p + n for n in live)
    else:
        new, lens = _extend_lengths(case, 1)
        w, s = case["window"], case["sinks"]
        rows, keys, pairs = sum(new), case["prefix"], 0
        for m, n in zip(new, lens):
            seen = [min(p + 1, w + min(s, max(0, p + 1 - w))) if w else p + 1 for p in range(n - m, n)]
            pairs += sum(seen)
            keys += min(n, m - 1 + w + s) if w else n - case["prefix"]
    return {"bytes": 2 * keys * hkv * dh * es + 2 * rows * hq * dh * es + 4 * rows * hq,
            "flops": 4 * pairs * hq * dh}


# ------------------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 5)
    rng = np.random.default_rng(seed * 104729 + 7)
    dt, hq, hkv, dh = DTYPES[case["dtype"]], case["hq"], case["hkv"], case["dh"]
    st = {"case": case, "scale": dh ** -0.5}
    if "sections" in case:
        n_axes = len(case["sections"].split(","))
        st["axis"] = torch.tensor(_axis_of(case)).cuda()
        st["inv_freq"] = torch.tensor(_frequencies(case), dtype=torch.float64).cuda()
        st["w_q"] = (1 + 0.2 * torch.randn(dh, generator=g, device="cuda")).to(dt)
        st["w_k"] = (1 + 0.2 * torch.randn(dh, generator=g, device="cuda")).to(dt)
    if case["op"] == "norm_axes":
        lead = (case["batch"], case["seqlen"]) if case["batch"] > 0 else (case["seqlen"],)
        # activations before a norm are not of unit size
        st["q"] = _randn(g, *lead, hq, dh, dtype=dt, scale=2.5)
        st["k"] = _randn(g, *lead, hkv, dh, dtype=dt, scale=2.5)
        st["dq_out"] = _randn(g, *lead, hq, dh, dtype=dt)
        st["dk_out"] = _randn(g, *lead, hkv, dh, dtype=dt)
        pos = np.concatenate([_axis_positions(n, n_axes, rng) for n in _lengths(case)])
        st["pos"] = torch.from_numpy(pos[_natural_rows(case)]).cuda().view(*lead, n_axes)
    elif case["op"] == "append_axes":
        new, old = _append_lengths(case, seed)
        n = sum(new)
        st["q"] = _randn(g, n, hq, dh, dtype=dt, scale=2.5)
        st["k"] = _randn(g, n, hkv, dh, dtype=dt, scale=2.5)
        st["v"] = _randn(g, n, hkv, dh, dtype=dt)
        st["new"] = torch.tensor(new).cuda()
        _offsets(st, new)
        pos = [o // 2 + _axis_positions(m, n_axes, rng) for m, o in zip(new, old)]
        st["pos"] = torch.from_numpy(np.concatenate(pos)).cuda()
        _pages(st, case, g, [a + b for a, b in zip(old, new)], [], [], fresh=True)
    elif case["op"] == "shared":
        starts, prefixes, mine = _shared_lengths(case, seed)
        st["q"] = _randn(g, case["batch"], hq, dh, dtype=dt)
        where = np.searchsorted(starts, np.arange(case["batch"]), side="right") - 1
        _pages(st, case, g, [prefixes[where[i]] + n if n >= 0 else 0 for i, n in enumerate(mine)],
               starts, prefixes)
    else:
        new, lens = _extend_lengths(case, seed)
        st["q"] = _randn(g, sum(new), hq, dh, dtype=dt)
        st["new"] = torch.tensor(new).cuda()
        _offsets(st, new)
        if case["groups"]:
            _pages(st, case, g, lens, [0, case["batch"]], [case["prefix"]])
        else:
            _pages(st, case, g, lens, [], [])
    if own:
        _handles(st, case)
    return st


def _offsets(st, new):
    st["cu_new"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32).cuda()


def _pages(st, case, g, lens, starts, prefixes, fresh=False):
    """A cache of pages in shuffled order, as after some hours of serving. The whole pages of a
    group's prefix are the same for all its sequences; a prefix that ends within a page goes on in
    a copy of that page for every sequence."""
    dt, page, b = DTYPES[case["dtype"]], case["page"], case["batch"]
    need = [-(-n // page) for n in lens]
    common = [0] * b
    for i, p in enumerate(prefixes):
        common[starts[i]:starts[i + 1]] = [p // page] * (starts[i + 1] - starts[i])
    # an append case returns its pages: as many for every seed, and nothing else in them
    total = 3 + (sum(-(-(n + case["old_max"]) // page) for n in st["new"].tolist()) if fresh
                 else sum(need) + sum(p // page for p in prefixes))
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(total)).int()
    span = max(case.get("max_len", 0), case.get("prefix", 0))  # the plain forms look a whole span up
    table = torch.zeros(b, max(need + [-(-span // page)]), dtype=torch.int32)
    at, copies = 0, []
    for i, p in enumerate(prefixes):
        m = p // page
        table[starts[i]:starts[i + 1], :m] = perm[at:at + m]
        at += m
    for i, n in enumerate(need):
        if n > common[i]:
            table[i, common[i]:n] = perm[at:at + n - common[i]]
            at += n - common[i]
    for i, p in enumerate(prefixes):
        live = [j for j in range(starts[i], starts[i + 1]) if need[j]]
        if p % page and live:
            first = table[live[0], p // page]
            copies += [(int(first), int(table[j, p // page])) for j in live[1:]]
            table[starts[i], p // page] = first  # (of an idle sequence too)
    shape = (total, page, case["hkv"], case["dh"])
    for x in ("k_pages", "v_pages"):
        st[x] = torch.zeros(shape, device="cuda", dtype=dt) if fresh else _randn(g, *shape, dtype=dt)
        if copies:
            src, dst = torch.tensor(copies).T.cuda()
            st[x][dst] = st[x][src]
    st["table"], st["lens"] = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    if prefixes:
        st["groups"] = torch.tensor(starts, dtype=torch.int32).cuda()
        st["prefixes"] = torch.tensor(prefixes, dtype=torch.int32).cuda()


def _handles(st, case):
    """What a user's program keeps next to its tensors: the problem, the rotation, the cache."""
    import context_blockwise_attention_step_gb300 as ra

    if case["op"] == "norm_axes":
        cu = None if case["batch"] > 0 else np.concatenate([[0], np.cumsum(_lengths(case))])
        st["prob"] = ra.problem_for(st["q"], st["k"], D=case["D"], layout=case["layout"],
                                    causal=True, cu_seqlens=cu)
    else:
        st["cache"] = ra.make_cache(st["k_pages"], st["v_pages"], st["table"])
    if "sections" in case:
        st["rope"] = ra.make_axis_rope(case["rotary"], _axis_of(case), inv_freq=_frequencies(case),
                                       interleaved=case["interleaved"])
    if "groups" in st:
        st["shared"] = ra.SharedPrefix(st["groups"], st["prefixes"])


# ------------------------------------------------------------------------------ run

def run(st):
    case = st["case"]
    if own:
        return _own(st, case)
    return {"norm_axes": _plain_norm_axes, "append_axes": _plain_append, "shared": _plain_shared,
            "extend": _plain_extend}[case["op"]](st, case)


def _own(st, case):
    import context_blockwise_attention_step_gb300 as ra

    if "sections" in case:
        how = dict(q_weight=st["w_q"], k_weight=st["w_k"], rope=st["rope"], positions=st["pos"], eps=EPS)
    if case["op"] == "norm_axes":
        q2, k2 = ra.qk_norm_rope_fwd(st["q"], st["k"], st["prob"], **how)
        dq, dk, dwq, dwk = ra.qk_norm_rope_bwd(st["dq_out"], st["dk_out"], st["q"], st["k"],
                                               st["prob"], **how)
        return {"q": q2, "k": k2, "dq": dq, "dk": dk, "dw_q": dwq, "dw_k": dwk}
    if case["op"] == "append_axes":
        cu_new = st["cu_new"] if case["new_max"] > 1 else None
        q2 = ra.kv_cache_append(st["q"], st["k"], st["v"], st["cache"], st["lens"], cu_new=cu_new, **how)
        return {"q": q2, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    if case["op"] == "shared":
        out, lse = ra.paged_attn_decode(st["q"], st["cache"], st["lens"], shared=st["shared"])
    else:
        out, lse = ra.paged_attn_extend(st["q"], st["cache"], st["lens"], st["cu_new"],
                                        shared=st.get("shared"), window=case["window"], sinks=case["sinks"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------------ plain forms

def _angles(st):
    pos = st["pos"].reshape(-1, st["pos"].shape[-1])[:, st["axis"]]
    a = pos.double() * st["inv_freq"]
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin, case):
    rd = case["rotary"]
    c, s, rest = cos[:, None], sin[:, None], x[..., rd:]
    if case["interleaved"]:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        both = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        both = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([both, rest], -1)


def _norm_rotate(x, w, cos, sin, case):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return _rotate(x * r * w.float(), cos, sin, case)


def _norm_rotate_back(dy, x, w, cos, sin, case):
    x, dy, w = x.float(), dy.float(), w.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    g = _rotate(dy, cos, -sin, case)
    n = x * r
    h = g * w
    dx = r * (h - n * (h * n).mean(-1, keepdim=True))
    return dx, (g * n).sum((0, 1), dtype=torch.float64).float()


def _plain_norm_axes(st, case):
    dt, dh = DTYPES[case["dtype"]], case["dh"]
    cos, sin = _angles(st)

    def one(x, w, grad):
        flat = x.reshape(-1, x.shape[-2], dh)
        y = _norm_rotate(flat, w, cos, sin, case)
        dx, dw = _norm_rotate_back(grad.reshape(flat.shape), flat, w, cos, sin, case)
        return y.to(dt).view(x.shape), dx.to(dt).view(x.shape), dw

    q, dq, dwq = one(st["q"], st["w_q"], st["dq_out"])
    k, dk, dwk = one(st["k"], st["w_k"], st["dk_out"])
    return {"q": q, "k": k, "dq": dq, "dk": dk, "dw_q": dwq, "dw_k": dwk}


def _token_rows(st):
    """Of every new token: its sequence and its place in it."""
    new, n = st["new"], st["q"].shape[0]
    seq = torch.repeat_interleave(torch.arange(new.numel(), device="cuda"), new, output_size=n)
    return seq, st["lens"].long()[seq] - new[seq] + torch.arange(n, device="cuda") - st["cu_new"].long()[seq]


def _plain_append(st, case):
    dt = DTYPES[case["dtype"]]
    seq, at = _token_rows(st)
    cos, sin = _angles(st)
    page, slot = st["table"][seq, at // case["page"]].long(), at % case["page"]
    st["k_pages"][page, slot] = _norm_rotate(st["k"], st["w_k"], cos, sin, case).to(dt)
    st["v_pages"][page, slot] = st["v"]
    return {"q": _norm_rotate(st["q"], st["w_q"], cos, sin, case).to(dt),
            "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _keys(st, case, table, span):
    """Keys and values 0 .. span - 1 of every row of a block table, in float32."""
    at = torch.arange(span, device="cuda")
    page, slot = table[:, at // case["page"]].long(), at % case["page"]
    return st["k_pages"][page, slot].float(), st["v_pages"][page, slot].float()


def _softmax_sums(s, v, how):
    """Row maximum, sum and weighted values of scores that are -inf where nothing is seen."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    return m, p.sum(-1, keepdim=True), torch.einsum(how, p, v)


def _result(m, total, out, case):
    """[.., heads, grp, 1] and [.., heads, grp, dh] into lse and out."""
    out = out / torch.where(total == 0, torch.ones_like(total), total)
    lse = (m + torch.log(total)).reshape(-1, case["hq"])
    return {"out": out.reshape(-1, case["hq"], case["dh"]).to(DTYPES[case["dtype"]]), "lse": lse}


def _plain_shared(st, case):
    """Every group's queries against its prefix, every query against its own keys, and both joined
    by their maxima and sums."""
    b, hkv, dh = case["batch"], case["hkv"], case["dh"]
    starts, prefixes, lens = st["groups"].long(), st["prefixes"].long(), st["lens"].long()
    n = prefixes.numel()
    where = torch.searchsorted(starts, torch.arange(b, device="cuda"), right=True) - 1
    member = torch.arange(b, device="cuda") - starts[where]
    q = st["q"].float().view(b, hkv, -1, dh) * st["scale"]
    qg = torch.zeros(n, b, hkv, q.shape[2], dh, device="cuda")
    qg[where, member] = q
    k, v = _keys(st, case, st["table"][starts[:-1]], case["prefix"])
    s = torch.einsum("nbhgd,nkhd->nbhgk", qg, k)
    at = torch.arange(case["prefix"], device="cuda")
    s = s.masked_fill_((at >= prefixes[:, None])[:, None, None, None], -math.inf)
    m1, l1, o1 = (x[where, member] for x in _softmax_sums(s, v, "nbhgk,nkhd->nbhgd"))
    mine = torch.arange(case["own_max"], device="cuda")[None] + prefixes[where][:, None]
    seen = mine < lens[:, None]
    mine = torch.where(seen, mine, torch.zeros_like(mine))
    page = torch.gather(st["table"].long(), 1, mine // case["page"])
    k, v = st["k_pages"][page, mine % case["page"]].float(), st["v_pages"][page, mine % case["page"]].float()
    s = torch.einsum("bhgd,bkhd->bhgk", q, k).masked_fill_(~seen[:, None, None], -math.inf)
    m2, l2, o2 = _softmax_sums(s, v, "bhgk,bkhd->bhgd")
    m = torch.maximum(m1, m2)
    live = (lens > 0)[:, None, None, None].float()
    f1, f2 = torch.exp(m1 - m) * live, torch.exp(m2 - m) * live
    return _result(m, l1 * f1 + l2 * f2, o1 * f1 + o2 * f2, case)


def _plain_extend(st, case):
    b, hkv, dh, span, most = case["batch"], case["hkv"], case["dh"], case["max_len"], case["new_max"]
    seq, pos = _token_rows(st)
    row = torch.arange(seq.numel(), device="cuda") - st["cu_new"].long()[seq]
    q = torch.zeros(b, most, hkv, case["hq"] // hkv, dh, device="cuda")
    q[seq, row] = st["q"].float().view(-1, *q.shape[2:]) * st["scale"]
    first = st["lens"].long() - st["new"]
    p = first[:, None, None] + torch.arange(most, device="cuda")[None, :, None]
    at = torch.arange(span, device="cuda")
    hidden = at > p
    if case["window"]:
        hidden |= (at <= p - case["window"]) & (at >= case["sinks"])
    k, v = _keys(st, case, st["table"], span)
    s = torch.einsum("bqhgd,bkhd->bqhgk", q, k).masked_fill_(hidden[:, :, None, None], -math.inf)
    m, total, out = (x[seq, row] for x in _softmax_sums(s, v, "bqhgk,bkhd->bqhgd"))
    return _result(m, total, out, case)


# ------------------------------------------------------------------------------ exact

def exact(case, seed):
    st = prepare(case, seed)
    return {"norm_axes": _exact_norm_axes, "append_axes": _exact_append, "shared": _exact_shared,
            "extend": _exact_extend}[case["op"]](st, case)


def _phases(st):
    """exp(i angle) of the rotated pairs of every token: [tokens, 1, pairs]."""
    p = st["pos"].reshape(-1, st["pos"].shape[-1]).double()
    angle = torch.stack([p[:, a] * f for a, f in zip(st["axis"].tolist(), st["inv_freq"])], -1)
    return torch.polar(torch.ones_like(angle), angle)[:, None]


def _turn(x, z, case):
    """The first ``rotary`` elements of every head as complex numbers, times z."""
    half, y = case["rotary"] // 2, x.clone()
    re, im = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (slice(0, half), slice(half, 2 * half))
    c = torch.complex(x[..., re], x[..., im]) * z
    y[..., re], y[..., im] = c.real, c.imag
    return y


def _exact_head(x, w, z, case):
    x = x.double()
    return _turn(x / ((x * x).mean(-1, keepdim=True) + EPS).sqrt() * w.double(), z, case)


def _exact_norm_axes(st, case):
    z_all, res = _phases(st), {}
    for x in ("q", "k"):
        flat, w = st[x].reshape(-1, *st[x].shape[-2:]), st["w_" + x].double()
        grad = st["d%s_out" % x].reshape(flat.shape)
        y, dx, dw = (torch.empty(flat.shape, dtype=torch.float64, device="cuda"),
                     torch.empty(flat.shape, dtype=torch.float64, device="cuda"), torch.zeros_like(w))
        for a in range(0, flat.shape[0], 16384):
            part, z = slice(a, a + 16384), z_all[a:a + 16384]
            y[part] = _exact_head(flat[part], w, z, case)
            v, back = flat[part].double(), _turn(grad[part].double(), z.conj(), case)
            ms = v.pow(2).mean(-1, keepdim=True) + EPS
            dw += (back * v / ms.sqrt()).sum((0, 1))
            back = back * w
            dx[part] = back / ms.sqrt() - v * (back * v).mean(-1, keepdim=True) / (ms * ms.sqrt())
        res[x], res["d" + x], res["dw_" + x] = y.view(st[x].shape), dx.view(st[x].shape), dw
    return res


def _exact_append(st, case):
    z = _phases(st)
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    k2 = _exact_head(st["k"], st["w_k"], z, case)
    cu, lens = st["cu_new"].tolist(), st["lens"].tolist()
    for b in range(case["batch"]):
        rows = slice(cu[b], cu[b + 1])
        at = torch.arange(lens[b] - (cu[b + 1] - cu[b]), lens[b], device="cuda")
        where = st["table"][b].long()[at // case["page"]], at % case["page"]
        kp[where], vp[where] = k2[rows], st["v"][rows].double()
    return {"q": _exact_head(st["q"], st["w_q"], z, case), "k_pages": kp, "v_pages": vp}


def _exact_rows(st, case, b, rows, q, first, out, lse):
    """Rows ``rows`` of the result: the queries q of sequence b at its places first, first + 1, ..."""
    hq, grp = case["hq"], case["hq"] // case["hkv"]
    n = first + q.shape[0]
    at = torch.arange(n, device="cuda")
    page, slot = st["table"][b].long()[at // case["page"]], at % case["page"]
    p = torch.arange(first, n, device="cuda")[:, None]
    seen = at <= p
    if case.get("window"):
        seen = seen & ((at > p - case["window"]) | (at < case["sinks"]))
    for h in range(hq):
        k, v = st["k_pages"][page, slot, h // grp].double(), st["v_pages"][page, slot, h // grp].double()
        for a in range(0, q.shape[0], 1024):
            part = slice(a, a + 1024)
            s = (q[part, h].double() @ k.T * st["scale"]).masked_fill_(~seen[part], -math.inf)
            l = torch.logsumexp(s, -1)
            lse[rows, h][part] = l
            out[rows, h][part] = torch.exp(s - l[:, None]) @ v


def _exact_shared(st, case):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        if n:
            _exact_rows(st, case, b, slice(b, b + 1), st["q"][b:b + 1], n - 1, out, lse)
    return {"out": out, "lse": lse}


def _exact_extend(st, case):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    cu = st["cu_new"].tolist()
    for b, n in enumerate(st["lens"].tolist()):
        rows = slice(cu[b], cu[b + 1])
        _exact_rows(st, case, b, rows, st["q"][rows], n - (cu[b + 1] - cu[b]), out, lse)
    return {"out": out, "lse": lse}
