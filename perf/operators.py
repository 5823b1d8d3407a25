"""Timed cases of the operators around ring attention: head norms with the position rotation,
the paged key-value cache with the attention that reads it, and sliding-window attention.

Each case is one pass through one operator:

  norm_rope  the queries and keys of a training step, natural or packed, in shard-major
             order: per-head root-mean-square norm and rotation, forward and backward
  append     new tokens of running sequences: norm and rotation of q and k, k and v written
             into the pages of the cache, the rotated q returned
  decode     attention of one new token of every sequence over the paged cache
  window     causal attention with a sliding window and a few always visible first tokens,
             over the shards of a ring layout, forward and backward

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
        # a short training batch: many small heads, where launches count
        dict(name="norm_rope_b2_s4096_h8_dh64", op="norm_rope", dtype="bf16", layout="basic", D=4,
             hq=8, hkv=8, dh=64, batch=2, seqlen=4096, n_seqs=0, rotary=64, interleaved=False),
        # one long context of a grouped-query model, forward and backward
        dict(name="norm_rope_s131072_gqa32x8_dh128", op="norm_rope", dtype="bf16", layout="zigzag",
             D=16, hq=32, hkv=8, dh=128, batch=1, seqlen=131072, n_seqs=0, rotary=128,
             interleaved=False),
        # the float32 path with packed sequences, an odd head size and a rotation of half of it
        dict(name="norm_rope_f32_varlen_dh96", op="norm_rope", dtype="f32", layout="stripe", D=8,
             hq=4, hkv=2, dh=96, batch=0, seqlen=8192, n_seqs=5, rotary=48, interleaved=True),
        # one decoding step of a small batch: latency
        dict(name="append_b4_decode", op="append", dtype="bf16", hq=32, hkv=8, dh=128, batch=4,
             new_max=1, old_max=4096, page=64, rotary=128, interleaved=False),
        # prompts of sixteen sequences of different lengths that go into the cache at once
        dict(name="append_16_prompts_s8192", op="append", dtype="bf16", hq=32, hkv=8, dh=128,
             batch=16, new_max=8192, old_max=100, page=64, rotary=128, interleaved=False),
        # interactive use: one sequence of some hundred tokens
        dict(name="decode_b1_s700", op="decode", dtype="bf16", hq=32, hkv=8, dh=128, batch=1,
             max_len=700, page=64, window=0, sinks=0),
        # one sequence of the long-context workload: all the work lies along the cache
        dict(name="decode_b1_s131072", op="decode", dtype="bf16", hq=32, hkv=8, dh=128, batch=1,
             max_len=131072, page=64, window=0, sinks=0),
        # a serving batch of ragged sequences, one of them idle
        dict(name="decode_b64_ragged_s16384", op="decode", dtype="bf16", hq=32, hkv=8, dh=128,
             batch=64, max_len=16384, page=64, window=0, sinks=0),
        # a model with a window: long caches of which little is read
        dict(name="decode_b33_window1024_sinks4_dh64", op="decode", dtype="bf16", hq=8, hkv=8,
             dh=64, batch=33, max_len=32768, page=16, window=1024, sinks=4),
        # short sequences of a training batch with a window shorter than a shard
        dict(name="window_b2_s4096_h8_dh64_w500", op="window", dtype="bf16", layout="basic", D=4,
             hq=8, hkv=8, dh=64, batch=2, seqlen=4096, n_seqs=0, window=500, sinks=4),
        # packed sequences of a grouped-query model
        dict(name="window_t65536_gqa32x8_w1024", op="window", dtype="bf16", layout="zigzag", D=8,
             hq=32, hkv=8, dh=128, batch=0, seqlen=65536, n_seqs=16, window=1024, sinks=4),
        # the float32 path
        dict(name="window_f32_s2048_dh64_w300", op="window", dtype="f32", layout="stripe", D=2,
             hq=4, hkv=2, dh=64, batch=1, seqlen=2048, n_seqs=0, window=300, sinks=2),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "decode", "decode", "window"])
    hq, hkv = rng.choice([(8, 8), (4, 2), (16, 16), (32, 8), (8, 1), (12, 4), (6, 2)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dh = rng.choice([64, 128]) if dtype == "bf16" else rng.choice([32, 48, 64, 96, 128])
    turned = dict(rotary=rng.choice([dh, dh // 2]), interleaved=rng.random() < 0.3)
    if op in ("norm_rope", "window"):
        D, layout = rng.choice([1, 2, 3, 4, 8]), rng.choice(["basic", "zigzag", "stripe"])
        most = {"norm_rope": (65536, 8192), "window": (32768, 1024)}[op][dtype == "f32"]
        n_seqs = rng.choice([0, 0, 3, 7, 16])
        batch = 0 if n_seqs else rng.choice([1, 2, 3])
        unit = 2 * D * max(1, batch)
        n = max(unit, _log_int(rng, 64, most) // unit * unit) // max(1, batch)
        c = dict(op=op, dtype=dtype, layout=layout, D=D, hq=hq, hkv=hkv, dh=dh, batch=batch,
                 seqlen=n, n_seqs=n_seqs)
        if op == "norm_rope":
            return dict(c, **turned)
        if dtype == "f32":
            c.update(hq=4, hkv=rng.choice([1, 2, 4]))
        return dict(c, window=_log_int(rng, 1, min(n, 1024)), sinks=rng.choice([0, 1, 4, 11]))
    page = rng.choice([16, 64, 128, 48])
    if op == "append":
        one = rng.random() < 0.5
        return dict(op=op, dtype=dtype, hq=hq, hkv=hkv, dh=dh, page=page,
                    batch=_log_int(rng, 1, 200) if one else rng.choice([1, 3, 16]),
                    new_max=1 if one else _log_int(rng, 2, 2900),
                    old_max=_log_int(rng, 1, 500), **turned)
    batch = _log_int(rng, 1, 128)
    max_len = _log_int(rng, 1, min(131072, 262144 // batch))
    w = rng.random() < 0.4
    return dict(op=op, dtype=dtype, hq=hq, hkv=hkv, dh=dh, batch=batch, max_len=max_len, page=page,
                window=_log_int(rng, 1, max_len) if w else 0,
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


def _shard_major(case):
    """Sequence, position and natural row of every shard-major row."""
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
            pieces[i, r] = pos
    order = ([(i, r) for i in range(len(lens)) for r in range(D)] if case["batch"] > 0
             else [(i, r) for r in range(D) for i in range(len(lens))])
    seq = np.concatenate([np.full(pieces[k].size, k[0], dtype=np.int64) for k in order])
    pos = np.concatenate([pieces[k] for k in order]).astype(np.int64)
    return seq, pos, starts[seq] + pos


def _serve_lengths(case, seed):
    """Lengths of the sequences of a decode case, from the seed: the first is the longest
    allowed, the others spread below it; from five sequences on, the last one is idle."""
    g = torch.Generator().manual_seed(seed * 1000003 + 17)
    b, hi = case["batch"], case["max_len"]
    lens = (1 + (torch.rand(b, generator=g) * hi).long()).clamp(max=hi)
    lens[0] = hi
    if b >= 5:
        lens[-1] = 0
    return lens


def _append_lengths(case, seed):
    """New tokens of each sequence (the same for every seed), and its tokens in the cache
    before them."""
    g = torch.Generator().manual_seed(seed * 1000003 + 19)
    new = torch.linspace(case["new_max"], 1, case["batch"]).long()
    old = (torch.rand(case["batch"], generator=g) * (case["old_max"] + 1)).long()
    return new, old


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, dh = case["hq"], case["hkv"], case["dh"]
    if case["op"] == "norm_rope":
        n = sum(_lengths(case)) * (hq + hkv) * dh
        return {"bytes": 5 * n * es + 2 * dh * es + 2 * dh * 4, "flops": 30 * n}
    if case["op"] == "append":
        n = int(_append_lengths(case, 1)[0].sum())
        return {"bytes": 2 * n * (hq + 2 * hkv) * dh * es + 8 * case["batch"],
                "flops": 10 * n * (hq + hkv) * dh}
    w, s = case["window"], case["sinks"]
    if case["op"] == "decode":
        keys, b, hi = 0.0, case["batch"], case["max_len"]
        for i in range(b):
            n = hi if i == 0 else 0 if b >= 5 and i == b - 1 else hi / 2  # the mean over seeds
            keys += n if not w or n <= w else w + min(s, n - w)
        return {"bytes": 2 * keys * hkv * dh * es + 2 * b * hq * dh * es + 4 * b * hq,
                "flops": 4 * keys * hq * dh}
    pairs, n = 0, sum(_lengths(case))
    for x in _lengths(case):
        m = min(x, w)
        far = x - m  # rows past the window: the i-th of them sees min(s, i + 1) more
        k = min(far, s)
        pairs += m * (m + 1) // 2 + far * w + k * (k + 1) // 2 + (far - k) * s
    # read: q, k, v, dO; written: out, lse, dq, dk, dv
    return {"bytes": (4 * hq + 4 * hkv) * n * dh * es + 4 * n * hq,
            "flops": 14 * pairs * hq * dh}


# ------------------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 5)
    dt, hq, hkv, dh = DTYPES[case["dtype"]], case["hq"], case["hkv"], case["dh"]
    st = {"case": case, "scale": dh ** -0.5}
    # activations before a norm are not of unit size
    size = 2.5 if "rotary" in case else 1.0
    if case["op"] in ("norm_rope", "window"):
        st["seq"], st["pos"], st["nat"] = (torch.from_numpy(x).cuda() for x in _shard_major(case))
        lead = (case["batch"], case["seqlen"]) if case["batch"] > 0 else (case["seqlen"],)
        st["q"] = _randn(g, *lead, hq, dh, dtype=dt, scale=size)
        st["k"] = _randn(g, *lead, hkv, dh, dtype=dt, scale=size)
        if case["op"] == "norm_rope":
            st["dq_out"] = _randn(g, *lead, hq, dh, dtype=dt)
            st["dk_out"] = _randn(g, *lead, hkv, dh, dtype=dt)
        else:
            st["v"] = _randn(g, *lead, hkv, dh, dtype=dt)
            st["dout"] = _randn(g, *lead, hq, dh, dtype=dt)
            lens = torch.tensor(_lengths(case))
            st["start"] = (torch.cumsum(lens, 0) - lens).cuda()
    elif case["op"] == "append":
        new, old = _append_lengths(case, seed)
        n = int(new.sum())
        st["q"] = _randn(g, n, hq, dh, dtype=dt, scale=size)
        st["k"] = _randn(g, n, hkv, dh, dtype=dt, scale=size)
        st["v"] = _randn(g, n, hkv, dh, dtype=dt)
        st["new"] = new.cuda()
        st["cu_new"] = torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(new, 0)]).int().cuda()
        _pages(st, case, g, old + new, case["old_max"] + case["new_max"])
    else:
        st["q"] = _randn(g, case["batch"], hq, dh, dtype=dt)
        _pages(st, case, g, _serve_lengths(case, seed), case["max_len"])
    if "rotary" in case:
        st["w_q"] = (1 + 0.2 * torch.randn(dh, generator=g, device="cuda")).to(dt)
        st["w_k"] = (1 + 0.2 * torch.randn(dh, generator=g, device="cuda")).to(dt)
        half = torch.arange(0, case["rotary"], 2, dtype=torch.float64) / case["rotary"]
        st["inv_freq"] = torch.pow(torch.tensor(BASE, dtype=torch.float64), -half).cuda()
    if own:
        _handles(st, case)
    return st


def _pages(st, case, g, lens, span):
    """A cache of pages in shuffled order, as after some hours of serving."""
    dt, page, b = DTYPES[case["dtype"]], case["page"], case["batch"]
    need = [(int(n) + page - 1) // page for n in lens]
    # an append case returns its pages: as many for every seed, and nothing else in them
    fresh = case["op"] == "append"
    total = 3 + (sum((int(n) + case["old_max"] + page - 1) // page for n in st["new"]) if fresh
                 else max(1, sum(need)))
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(total)).int()
    table = torch.zeros(b, (span + page - 1) // page, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    shape = (total, page, case["hkv"], case["dh"])
    for x in ("k_pages", "v_pages"):
        st[x] = torch.zeros(shape, device="cuda", dtype=dt) if fresh else _randn(g, *shape, dtype=dt)
    st["table"], st["lens"] = table.cuda(), lens.int().cuda()


def _handles(st, case):
    """What a user's program keeps next to its tensors: the problem, the rotation, the cache."""
    import context_blockwise_attention_step_gb300 as ra

    if case["op"] in ("norm_rope", "window"):
        cu = None if case["batch"] > 0 else np.concatenate([[0], np.cumsum(_lengths(case))])
        st["prob"] = ra.problem_for(st["q"], st["k"], D=case["D"], layout=case["layout"],
                                    causal=True, cu_seqlens=cu)
    else:
        st["cache"] = ra.make_cache(st["k_pages"], st["v_pages"], st["table"])
    if "rotary" in case:
        st["rope"] = ra.make_rope(case["rotary"], inv_freq=st["inv_freq"].cpu().tolist(),
                                  interleaved=case["interleaved"])


# ------------------------------------------------------------------------------ run

def run(st):
    case = st["case"]
    if own:
        return _own(st, case)
    return {"norm_rope": _plain_norm_rope, "append": _plain_append, "decode": _plain_decode,
            "window": _plain_window}[case["op"]](st, case)


def _own(st, case):
    import context_blockwise_attention_step_gb300 as ra

    if case["op"] == "norm_rope":
        how = dict(q_weight=st["w_q"], k_weight=st["w_k"], rope=st["rope"], eps=EPS)
        q2, k2 = ra.qk_norm_rope_fwd(st["q"], st["k"], st["prob"], **how)
        dq, dk, dwq, dwk = ra.qk_norm_rope_bwd(st["dq_out"], st["dk_out"], st["q"], st["k"],
                                               st["prob"], **how)
        return {"q": q2, "k": k2, "dq": dq, "dk": dk, "dw_q": dwq, "dw_k": dwk}
    if case["op"] == "append":
        cu_new = st["cu_new"] if case["new_max"] > 1 else None
        q2 = ra.kv_cache_append(st["q"], st["k"], st["v"], st["cache"], st["lens"], cu_new=cu_new,
                                q_weight=st["w_q"], k_weight=st["w_k"], rope=st["rope"], eps=EPS)
        return {"q": q2, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    how = dict(window=case["window"], sinks=case["sinks"])
    if case["op"] == "decode":
        out, lse = ra.paged_attn_decode(st["q"], st["cache"], st["lens"], **how)
        return {"out": out, "lse": lse}
    q, k, v, prob = st["q"], st["k"], st["v"], st["prob"]
    out, lse = ra.window_attn_fwd(q, k, v, prob, **how)
    dq, dk, dv = ra.window_attn_bwd(st["dout"], q, k, v, out, lse, prob, **how)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# ------------------------------------------------------------------------------ plain forms

def _angles(pos, inv_freq):
    a = pos.double()[:, None] * inv_freq[None, :]
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


def _plain_norm_rope(st, case):
    dt, res = DTYPES[case["dtype"]], {}
    cos, sin = _angles(st["pos"], st["inv_freq"])
    for x in ("q", "k"):
        flat, w = st[x].reshape(-1, *st[x].shape[-2:]), st["w_" + x]
        grad = st["d%s_out" % x].reshape(flat.shape)
        res[x] = _norm_rotate(flat, w, cos, sin, case).to(dt).view(st[x].shape)
        dx, res["dw_" + x] = _norm_rotate_back(grad, flat, w, cos, sin, case)
        res["d" + x] = dx.to(dt).view(st[x].shape)
    return res


def _plain_append(st, case):
    dt, new, n = DTYPES[case["dtype"]], st["new"], st["q"].shape[0]
    seq = torch.repeat_interleave(torch.arange(case["batch"], device="cuda"), new, output_size=n)
    within = torch.arange(n, device="cuda") - st["cu_new"].long()[seq]
    pos = st["lens"].long()[seq] - new[seq] + within
    cos, sin = _angles(pos, st["inv_freq"])
    page, slot = st["table"][seq, pos // case["page"]].long(), pos % case["page"]
    st["k_pages"][page, slot] = _norm_rotate(st["k"], st["w_k"], cos, sin, case).to(dt)
    st["v_pages"][page, slot] = st["v"]
    return {"q": _norm_rotate(st["q"], st["w_q"], cos, sin, case).to(dt),
            "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _plain_decode(st, case):
    dt, b, hkv = DTYPES[case["dtype"]], case["batch"], case["hkv"]
    lens = st["lens"].long()[:, None]
    keys = torch.arange(case["max_len"], device="cuda")[None, :]
    seen = keys < lens
    if case["window"]:
        seen = seen & ((keys >= lens - case["window"]) | (keys < case["sinks"]))
    page = st["table"][:, keys[0] // case["page"]].long()
    k = st["k_pages"][page, keys % case["page"]].float()
    v = st["v_pages"][page, keys % case["page"]].float()
    q = st["q"].float().view(b, hkv, -1, case["dh"])
    s = torch.einsum("bhgd,bkhd->bhgk", q, k) * st["scale"]
    s = s.masked_fill(~seen[:, None, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bhgk,bkhd->bhgd", p, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (m + torch.log(total)).view(b, -1)
    return {"out": out.reshape(b, -1, case["dh"]).to(dt), "lse": lse}


def _plain_window(st, case):
    """Blocks of queries against the band of keys that some query of the block may see, and
    every query against the first tokens of its sequence."""
    dt, w, sinks, hq, hkv, dh = (DTYPES[case["dtype"]], case["window"], case["sinks"], case["hq"],
                                 case["hkv"], case["dh"])
    n, grp, blk = st["nat"].numel(), hq // hkv, 256
    nb = -(-n // blk)
    pad = nb * blk - n
    order = torch.empty_like(st["nat"])  # natural order
    order[st["nat"]] = torch.arange(n, device="cuda")
    q, k, v, do = (st[x].reshape(n, -1, dh)[order].float() for x in ("q", "k", "v", "dout"))
    seq, pos = st["seq"][order], st["pos"][order]
    fill = torch.nn.functional.pad

    def blocks(x):  # [n, hq, dh] -> [nb, blk, hkv, grp, dh]
        return fill(x, (0, 0, 0, 0, 0, pad)).view(nb, blk, hkv, grp, dh)

    def rows(x):  # [nb, hkv, grp, blk] -> [n, hkv, grp]
        return x.permute(0, 3, 1, 2).reshape(nb * blk, hkv, grp)[:n]

    def per_score(x):  # [n, hkv, grp] -> [nb, hkv, grp, blk, 1]
        return fill(x, (0, 0, 0, 0, 0, pad)).view(nb, blk, hkv, grp).permute(0, 2, 3, 1)[..., None]

    def unblock(x):  # [nb, blk, hkv, grp, dh] -> [n, hkv, grp, dh]
        return x.reshape(nb * blk, hkv, grp, dh)[:n]

    # the band: the keys from first - w + 1 to first + blk - 1 of every block
    at = (torch.arange(nb, device="cuda") * blk - (w - 1))[:, None] + torch.arange(blk + w - 1, device="cuda")
    inside = (at >= 0) & (at < n)
    at = at.clamp(0, n - 1)
    seq_q, pos_q = fill(seq, (0, pad), value=-1).view(nb, blk, 1), fill(pos, (0, pad)).view(nb, blk, 1)
    seq_k, pos_k = seq[at][:, None, :], pos[at][:, None, :]
    seen = inside[:, None, :] & (seq_k == seq_q) & (pos_k <= pos_q) & (pos_k > pos_q - w)
    hidden = ~seen[:, None, None]
    qb, dob, kb, vb = blocks(q), blocks(do), k[at], v[at]
    s = torch.einsum("nqhgd,nkhd->nhgqk", qb, kb) * st["scale"]
    s = s.masked_fill_(hidden, -math.inf)
    # the first tokens of the sequence, as far as they lie before the window
    place = torch.arange(max(sinks, 1), device="cuda")[None, :]
    sink_at = (st["start"][seq][:, None] + place).clamp(max=n - 1)
    sink_seen = (place < sinks) & (place <= pos[:, None] - w)
    ks, vs = k[sink_at], v[sink_at]  # [n, sinks, hkv, dh]
    qg, dog = q.view(n, hkv, grp, dh), do.view(n, hkv, grp, dh)
    z = torch.einsum("nhgd,nkhd->nhgk", qg, ks) * st["scale"]
    z = z.masked_fill(~sink_seen[:, None, None], -math.inf)
    m = torch.maximum(rows(s.amax(-1)), z.amax(-1))
    p = torch.exp(s - per_score(m)).masked_fill_(hidden, 0.0)
    pz = torch.exp(z - m[..., None])
    total = rows(p.sum(-1)) + pz.sum(-1)
    p = p / per_score(total).clamp(min=1e-30)
    pz = pz / total[..., None]
    out = unblock(torch.einsum("nhgqk,nkhd->nqhgd", p, vb)) + torch.einsum("nhgk,nkhd->nhgd", pz, vs)
    lse = m + torch.log(total)
    # backward: dS = P * (dO V^T - rowsum(dO * O))
    delta = (dog * out).sum(-1)
    ds = p * (torch.einsum("nqhgd,nkhd->nhgqk", dob, vb) - per_score(delta))
    dz = pz * (torch.einsum("nhgd,nkhd->nhgk", dog, vs) - delta[..., None])
    dq = unblock(torch.einsum("nhgqk,nkhd->nqhgd", ds, kb)) + torch.einsum("nhgk,nkhd->nhgd", dz, ks)

    def keys_of(band, far):
        to = torch.zeros(n, hkv, dh, device="cuda")
        to.index_add_(0, at.reshape(-1), band.reshape(-1, hkv, dh))
        return to.index_add_(0, sink_at.reshape(-1), far.reshape(-1, hkv, dh))

    dv = keys_of(torch.einsum("nhgqk,nqhgd->nkhd", p, dob), torch.einsum("nhgk,nhgd->nkhd", pz, dog))
    dk = keys_of(torch.einsum("nhgqk,nqhgd->nkhd", ds, qb), torch.einsum("nhgk,nhgd->nkhd", dz, qg))

    def back(x, like):
        return x.reshape(n, -1, dh)[st["nat"]].to(dt).view(like.shape)

    return {"out": back(out, st["q"]), "lse": _lse_layout(lse.reshape(n, hq)[st["nat"]], case),
            "dq": back(dq * st["scale"], st["q"]), "dk": back(dk * st["scale"], st["k"]),
            "dv": back(dv, st["k"])}


def _lse_layout(lse, case):
    """[rows, hq] -> [batch, hq, seqlen], or [hq, rows] of packed sequences."""
    if case["batch"] > 0:
        return lse.view(case["batch"], -1, case["hq"]).transpose(1, 2).contiguous()
    return lse.t().contiguous()


# ------------------------------------------------------------------------------ exact

def exact(case, seed):
    st = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "append": _exact_append, "decode": _exact_decode,
            "window": _exact_window}[case["op"]](st, case)


def _phases(pos, inv_freq):
    a = pos.double()[:, None] * inv_freq[None, :]
    return torch.polar(torch.ones_like(a), a)


def _turn(x, z, case):
    """x [n, h, dh] with its pairs, read as complex numbers, multiplied by z [n, rotary / 2]."""
    x, rd = x.clone(), case["rotary"]
    first, second = ((slice(0, rd, 2), slice(1, rd, 2)) if case["interleaved"]
                     else (slice(0, rd // 2), slice(rd // 2, rd)))
    c = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * z[:, None]
    x[..., first], x[..., second] = c.real, c.imag
    return x


def _exact_head(x, w, z, case):
    x = x.double()
    return _turn(x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * w.double(), z, case)


def _exact_norm_rope(st, case):
    z_all = _phases(st["pos"], st["inv_freq"])
    res = {}
    for x in ("q", "k"):
        flat, w = st[x].reshape(-1, *st[x].shape[-2:]), st["w_" + x].double()
        grad = st["d%s_out" % x].reshape(flat.shape)
        y = torch.empty(flat.shape, dtype=torch.float64, device="cuda")
        dx, dw = torch.empty_like(y), torch.zeros_like(w)
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
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    q2 = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    cu, lens, table = st["cu_new"].tolist(), st["lens"].tolist(), st["table"].long()
    for b in range(case["batch"]):
        rows = slice(cu[b], cu[b + 1])
        pos = torch.arange(lens[b] - (cu[b + 1] - cu[b]), lens[b], device="cuda")
        z = _phases(pos, st["inv_freq"])
        q2[rows] = _exact_head(st["q"][rows], st["w_q"], z, case)
        where = table[b][pos // case["page"]], pos % case["page"]
        kp[where] = _exact_head(st["k"][rows], st["w_k"], z, case)
        vp[where] = st["v"][rows].double()
    return {"q": q2, "k_pages": kp, "v_pages": vp}


def _exact_decode(st, case):
    b, hq, grp = case["batch"], case["hq"], case["hq"] // case["hkv"]
    out = torch.zeros(b, hq, case["dh"], dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    table = st["table"].long()
    for i, n in enumerate(st["lens"].tolist()):
        pos = torch.arange(n, device="cuda")
        if case["window"]:
            pos = pos[(pos > n - 1 - case["window"]) | (pos < case["sinks"])]
        page, slot = table[i][pos // case["page"]], pos % case["page"]
        k, v = st["k_pages"][page, slot].double(), st["v_pages"][page, slot].double()
        for h in range(hq if n else 0):
            s = (k[:, h // grp] @ st["q"][i, h].double()) * st["scale"]
            lse[i, h] = torch.logsumexp(s, 0)
            out[i, h] = torch.softmax(s, 0) @ v[:, h // grp]
    return {"out": out, "lse": lse}


def _exact_window(st, case):
    w, sinks, hq, hkv, dh = case["window"], case["sinks"], case["hq"], case["hkv"], case["dh"]
    n, grp, scale = st["nat"].numel(), hq // hkv, st["scale"]
    order = torch.argsort(st["nat"])
    q, k, v, do = (st[x].reshape(n, -1, dh)[order].double() for x in ("q", "k", "v", "dout"))
    out, dq = torch.zeros_like(q), torch.zeros_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.zeros(n, hq, dtype=torch.float64, device="cuda")
    step, start = 1024, 0
    for length in _lengths(case):
        for a in range(0, length, step):
            p = torch.arange(a, min(length, a + step), device="cuda")
            lo = max(0, a - w + 1)
            keys = torch.cat([torch.arange(0, min(sinks, lo), device="cuda"),
                              torch.arange(lo, min(length, a + step), device="cuda")])
            ok = (keys[None] <= p[:, None]) & ((keys[None] > p[:, None] - w) | (keys[None] < sinks))
            r, c = start + p, start + keys
            for h in range(hkv):
                hs = slice(h * grp, (h + 1) * grp)
                qq, dd = q[r, hs].transpose(0, 1), do[r, hs].transpose(0, 1)  # [grp, rows, dh]
                kk, vv = k[c, h], v[c, h]
                s = (qq @ kk.T * scale).masked_fill(~ok, -math.inf)
                l = torch.logsumexp(s, -1)
                pr = torch.exp(s - l[..., None])
                o = pr @ vv
                g = pr * (dd @ vv.T - (dd * o).sum(-1, keepdim=True))
                out[r, hs], lse[r, hs] = o.transpose(0, 1), l.t()
                dq[r, hs] = (g @ kk * scale).transpose(0, 1)
                dv[c, h] += (pr.transpose(1, 2) @ dd).sum(0)
                dk[c, h] += (g.transpose(1, 2) @ qq).sum(0) * scale
        start += length

    def back(x, like):
        return x[st["nat"]].view(like.shape)

    return {"out": back(out, st["q"]), "lse": _lse_layout(lse[st["nat"]], case),
            "dq": back(dq, st["q"]), "dk": back(dk, st["k"]), "dv": back(dv, st["k"])}
