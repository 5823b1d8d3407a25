"""The calls of the attention of several new tokens over a paged cache as programs make them: on other
streams, captured, with used workspaces, two at once, over long caches, with what may not be followed; and
the operators together, in the layer.

Tolerances as in test_gpu_extend.py; repeats of a call give the same bits.
"""
import numpy as np
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from context_blockwise_attention_step_gb300 import _abi
from oracle import heads as H
from test_gpu_extend import BIG, Batch, f64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def two_batches():
    """One token each behind two shared prefixes, and several tokens behind one, of few and many rows."""
    one = Batch(3, BF16, 16, 4, 64, 16, [705, 701, 730, 305, 301, 0, 40], groups=[(3, 700), (3, 300), (1, 0)], capacity=BIG)
    lens, news = [900, 803, 990, 801, 870], [100, 3, 190, 1, 70]
    many = Batch(4, BF16, 8, 2, 128, 64, lens, news, groups=[(5, 800)], capacity=BIG)
    return one, many


def test_streams_graphs_and_workspaces():
    for b, how in zip(two_batches(), ({"cu_new": None}, {})):
        want = b.run(**how)
        b.check(*want)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = b.run(stream=s, **how)
        s.synchronize()
        assert same(got, want)
        n = ra.paged_extend_workspace_bytes(b.cache, b.q.shape[0], b.hq, b.shared)
        ws = torch.full((n,), 0xFF, device="cuda", dtype=torch.uint8)
        out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.run(workspace=ws, out=out, lse=lse, **how)
        for fill in (0xFF, 0x00, 0x7F):
            ws.fill_(fill)
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert same((out, lse), want)
        # the lengths are read when the graph runs: every sequence idle, and back
        if not how:
            continue
        keep = b.seq_lens.clone()
        b.seq_lens.zero_()
        graph.replay()
        assert (out == 0).all() and torch.isneginf(lse).all()
        b.seq_lens.copy_(keep)
        graph.replay()
        assert same((out, lse), want)
    assert ra.check_device_status() == _abi.RA_OK, ra.last_error()


def test_two_calls_at_once():
    """On two streams, with workspaces of their own, many times over: the same bits."""
    one, many = two_batches()
    want = one.run(cu_new=None), many.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(10):
        got.append((one.run(cu_new=None, stream=s1), many.run(stream=s2)))
    torch.cuda.synchronize()
    for a, b in got:
        assert same(a, want[0]) and same(b, want[1])
    assert ra.check_device_status() == _abi.RA_OK, ra.last_error()


@pytest.mark.parametrize("order", ["phsd", "wide"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
def test_orders_of_the_pages(order, dtype):
    """Heads before places, and keys and values side by side in one tensor."""
    b = Batch(5, dtype, 8, 4, 64, 16, [300, 40, 131], [200, 2, 5], order=order)
    b.check(*b.run())
    lens = [516, 530, 513]
    b = Batch(6, dtype, 8, 4, 64, 16, lens, groups=[(3, 512)], order=order, capacity=BIG)
    b.check(*b.run(cu_new=None))


def test_rows_of_no_sequence_are_left_as_they_are():
    for dtype, dh in ((BF16, 64), (F32, 40)):
        b = Batch(7, dtype, 4, 2, dh, 16, [50, 300], [20, 130])
        want = b.run()
        pad = 5
        q = torch.cat([torch.full_like(b.q[:pad], float("nan")), b.q, torch.full_like(b.q[:pad], float("nan"))])
        out, lse = torch.full_like(q, 7.0), torch.full((q.shape[0], 4), 7.0, device="cuda")
        ra.paged_attn_extend(q, b.cache, b.seq_lens, b.cu_new + pad, out=out, lse=lse)
        assert same((out[pad:-pad], lse[pad:-pad]), want)
        for t in (out, lse):
            assert (t[:pad] == 7).all() and (t[-pad:] == 7).all()
        assert ra.check_device_status() == _abi.RA_OK, ra.last_error()


def test_groups_that_share_nothing_in_the_end():
    """A prefix that a sequence does not have before its new tokens, one longer than the table, sequences of
    no group, an idle first sequence with nothing in its table: the same results."""
    lens = [0, 700, 650, 640, 900, 33]
    b = Batch(8, BF16, 8, 2, 64, 16, lens, groups=[(4, 640), (2, 0)], capacity=BIG)  # 640 with the new token
    ref = b.reference()
    b.check(*b.run(cu_new=None), ref)
    for prefix in ([639, 0], [1 << 30, 5], [-3, 0], [600, 33]):
        shared = ra.SharedPrefix(b.shared.cu_groups, torch.tensor(prefix, dtype=torch.int32).cuda())
        if prefix[0] == 600 or prefix[0] < 640:  # (what a group shares has to be equal)
            b.check(*b.run(cu_new=None, shared=shared), ref, str(prefix))
    part = ra.SharedPrefix(torch.tensor([1, 4], dtype=torch.int32).cuda(), torch.tensor([600], dtype=torch.int32).cuda())
    b.check(*b.run(cu_new=None, shared=part), ref, "some sequences in no group")


def test_what_may_not_be_followed_is_recorded():
    b = Batch(9, BF16, 8, 2, 64, 16, [300, 200, 100, 50], [30, 20, 10, 5])
    want = b.run()
    assert ra.check_device_status() == _abi.RA_OK

    def run(seq_lens=None, cu=None, cache=None):
        out, lse = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
        ra.paged_attn_extend(b.q, cache or b.cache, b.seq_lens if seq_lens is None else seq_lens,
                             b.cu_new if cu is None else torch.tensor(cu, dtype=torch.int32).cuda(), out=out, lse=lse)
        assert ra.check_device_status() == _abi.RA_ERR_CACHE_INDEX
        assert ra.check_device_status() == _abi.RA_OK
        return out, lse
    lens = b.seq_lens.clone()
    lens[2] = 3  # fewer than its new tokens: its rows see nothing
    out, lse = run(lens)
    assert (out[50:60] == 0).all() and torch.isneginf(lse[50:60]).all()
    assert same((out[:50], lse[:50]), (want[0][:50], want[1][:50])) and same((out[60:], lse[60:]), (want[0][60:], want[1][60:]))
    lens[2] = -5
    out, lse = run(lens)
    assert (out[50:60] == 0).all() and same((out[60:], lse[60:]), (want[0][60:], want[1][60:]))
    out, lse = run(cu=[0, 30, 50, 60, 1000])  # past the rows
    assert same((out[:60], lse[:60]), (want[0][:60], want[1][:60]))
    run(cu=[0, 30, 20, 60, 65])               # decreasing
    run(cu=[-7, 30, 50, 60, 65])
    table = b.table.clone()
    table[1, 3] = b.pages[0].shape[0]
    out, lse = run(cache=ra.make_cache(*b.pages, table))
    rows = slice(50, 65)
    assert same((out[rows], lse[rows]), (want[0][rows], want[1][rows]))
    with pytest.raises(ra.RingAttnError):
        ra.paged_attn_extend(b.q, b.cache, b.seq_lens, b.cu_new, shared=two_batches()[0].shared, window=5)
    with pytest.raises(ValueError):
        ra.paged_attn_extend(b.q, b.cache, b.seq_lens, b.cu_new.long())
    with pytest.raises(ValueError):
        ra.paged_attn_extend(b.q.transpose(0, 1).contiguous().transpose(0, 1), b.cache, b.seq_lens, b.cu_new)


def test_layer_refuses_positions_without_axes():
    x, at = torch.zeros(1, 64, 32, device="cuda", dtype=BF16), torch.zeros(1, 64, 2, device="cuda", dtype=torch.int32)
    for kw in (dict(), dict(rope=ra.make_rope(64)), dict(qk_norm=True)):
        with pytest.raises(ValueError):
            ra.RingSelfAttention(32, 2, 1, 64, D=1, layout="basic", device="cuda", **kw)(x, at)


def dense(b, rows, seq, first):
    """out and lse of some rows of sequence `seq`, in float64 on the GPU."""
    n = first + (rows.stop - rows.start)
    at = torch.arange(n, device="cuda")
    page, slot = b["table"][seq].long()[at // b["page"]], at % b["page"]
    k, v = (b[x][page, slot].double() for x in ("k", "v"))
    q = b["q"][rows].double()
    grp = q.shape[1] // k.shape[1]
    s = torch.einsum("rhgd,khd->rhgk", q.view(q.shape[0], -1, grp, q.shape[2]), k) * q.shape[2] ** -0.5
    s = s.masked_fill((at > torch.arange(first, n, device="cuda")[:, None])[:, None, None], -float("inf"))
    p = torch.softmax(s, -1)
    o, mag = (torch.einsum("rhgk,khd->rhgd", p, x).reshape(q.shape) for x in (v, v.abs()))
    return o, torch.logsumexp(s, -1).reshape(q.shape[:2]), mag


@pytest.mark.parametrize("dtype,hq,hkv,dh,prefix,own,news", [
    (BF16, 12, 1, 64, 100000, [3, 1, 40], None),         # one K/V head: every CTA has a part of a row
    (BF16, 6, 6, 128, 30000, [1, 2], None),              # two rows a K/V head behind the prefix
    (BF16, 8, 1, 128, 20011, [300, 5, 130], [256, 5, 1]),
    (F32, 8, 1, 64, 20000, [3, 1, 40, 2], None),
    (F32, 3, 1, 128, 9000, [70, 3], [65, 1]),
], ids=str)
def test_long_prefixes(dtype, hq, hkv, dh, prefix, own, news):
    page, n = 64, len(own)
    need = [-(-(prefix + m) // page) for m in own]
    shared, total = prefix // page, prefix // page + sum(x - prefix // page for x in need)
    g = torch.Generator(device="cuda").manual_seed(11)
    b = {"page": page}
    for x in ("k", "v"):
        b[x] = torch.randn(total, page, hkv, dh, generator=g, device="cuda").to(dtype)
    table = torch.zeros(n, max(max(need), BIG // (n * page * hkv * dh * 4)), dtype=torch.int32)
    at = shared
    for i, m in enumerate(need):
        table[i, :shared] = torch.arange(shared)
        table[i, shared:m] = torch.arange(at, at + m - shared)
        at += m - shared
        if i and prefix % page:  # the tokens of the page in which the prefix ends are the same as well
            for x in ("k", "v"):
                b[x][table[i, shared], :prefix % page] = b[x][table[0, shared], :prefix % page]
    b["table"] = table.cuda()
    new = [1] * n if news is None else news
    cu = np.concatenate([[0], np.cumsum(new)])
    b["q"] = (torch.randn(cu[-1], hq, dh, generator=g, device="cuda") * 1.5).to(dtype)
    cache = ra.make_cache(b["k"], b["v"], b["table"])
    lens = torch.tensor([prefix + m for m in own], dtype=torch.int32).cuda()
    how = dict(shared=ra.SharedPrefix(torch.tensor([0, n], dtype=torch.int32).cuda(), torch.tensor([prefix], dtype=torch.int32).cuda()),
               cu_new=None if news is None else torch.from_numpy(cu).int().cuda())
    out, lse = ra.paged_attn_extend(b["q"], cache, lens, **how)
    assert ra.check_device_status() == _abi.RA_OK, ra.last_error()
    half = 2.0 ** -8 if dtype == BF16 else 0.0
    for i in range(n):
        rows = slice(int(cu[i]), int(cu[i + 1]))
        o, l, mag = dense(b, rows, i, prefix + own[i] - new[i])
        assert ((out[rows] - o).abs() <= (half + 2.0 ** -11) * mag + half * o.abs()).all(), f"out of sequence {i}"
        assert ((lse[rows] - l).abs() <= 2.0 ** -12 + 2.0 ** -22 * l.abs()).all(), f"lse of sequence {i}"
    assert same((out, lse), ra.paged_attn_extend(b["q"], cache, lens, **how))


def test_pages_past_32_bits():
    """Pages whose elements lie more than 2^31 elements behind the first."""
    hkv, dh, page = 2, 128, 16
    far = (1 << 31) // (page * hkv * dh) + 7  # pages
    k, v = (torch.empty((far + 20) * page * hkv * dh, device="cuda", dtype=BF16).view(-1, page, hkv, dh) for _ in range(2))
    lens, news = [250, 130], [100, 3]
    b = Batch(12, BF16, 8, hkv, dh, page, lens, news)
    table = b.table.clone()
    for i, m in enumerate(lens):
        for j in range(-(-m // page)):
            table[i, j] = far - 5 + i * 10 + j if j < 10 else j
            for dst, src in ((k, b.pages[0]), (v, b.pages[1])):
                dst[table[i, j]] = src[b.table[i, j]]
    table[1, 5:9] = torch.tensor([far + 15, far + 16, far + 17, far + 18], dtype=torch.int32)
    for j in range(5, 9):
        k[table[1, j]], v[table[1, j]] = b.pages[0][b.table[1, j]], b.pages[1][b.table[1, j]]
    want = b.run()
    got = ra.paged_attn_extend(b.q, ra.make_cache(k, v, table), b.seq_lens, b.cu_new)
    assert same(got, want)
    assert ra.check_device_status() == _abi.RA_OK, ra.last_error()


# ------------------------------------------------------------------------------ the layer

TOL = 2.0 ** -6.5  # six independent roundings to bf16 on a token's way through the layer, relative L2
AXIS = ra.axis_sections([8, 12, 12])


def layer(window=0, sinks=0, axes=True, **kw):
    rope = ra.make_axis_rope(64, AXIS) if axes else ra.make_rope(64)
    m = ra.RingSelfAttention(96, 8, 2, 64, device="cuda", seed=5, qk_norm=True, window=window, sinks=sinks, rope=rope,
                             **{"D": 2, "layout": "zigzag", **kw})
    with torch.no_grad():
        g = torch.Generator().manual_seed(6)
        for w in (m.q_norm, m.k_norm):
            w.copy_(1 + 0.3 * torch.randn(64, generator=g))
    return m


def places(n, seed):
    """Positions of n tokens on three axes: text, then an image, then text."""
    rng = np.random.default_rng(seed)
    p = np.repeat(np.arange(n)[:, None], 3, 1)
    a = min(n, 20)
    i = np.arange(n - a)
    p[a:] = a + np.stack([i * 0, i // 9, i % 9], -1)
    return (p + rng.integers(0, 3)).astype(np.int32)


def reference(m, X, P, GY=None):
    W = {n: f64(p) for n, p in m.named_parameters()}
    n = X.shape[0]
    z = H.axis_phases(P, AXIS, 10000.0 ** (-np.arange(0, 64, 2) / 64))
    q0, k0 = (X @ W["wq"].T).reshape(n, 8, -1), (X @ W["wk"].T).reshape(n, 2, -1)
    v = (X @ W["wv"].T).reshape(n, 2, -1)
    q, k = (H.norm_rope_fwd(t, W[w], z, m.eps) for t, w in ((q0, "q_norm"), (k0, "k_norm")))
    ok, scale = H.seen(n, n, m.window, m.sinks), 64 ** -0.5
    out, _ = H.masked_fwd(q, k, v, ok, scale)
    if GY is None:
        return out.reshape(n, -1) @ W["wo"].T
    dq, dk, dv = H.masked_bwd(q, k, v, (GY @ W["wo"]).reshape(out.shape), ok, scale)
    dq, dqn = H.norm_rope_bwd(dq, q0, W["q_norm"], z, m.eps)
    dk, dkn = H.norm_rope_bwd(dk, k0, W["k_norm"], z, m.eps)
    flat = lambda t: t.reshape(n, -1)  # noqa: E731
    return {"x": flat(dq) @ W["wq"] + flat(dk) @ W["wk"] + flat(dv) @ W["wv"], "wq": flat(dq).T @ X, "wk": flat(dk).T @ X,
            "wv": flat(dv).T @ X, "wo": GY.T @ flat(out), "q_norm": dqn, "k_norm": dkn}


def rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


@pytest.mark.parametrize("kw", [dict(), dict(layout="stripe", window=50, sinks=3), dict(shard_major=True)], ids=str)
def test_layer_with_axes_output_and_gradients(kw):
    m = layer(**kw)
    g = torch.Generator().manual_seed(7)
    x = torch.randn(1, 300, 96, generator=g).cuda().bfloat16()
    gy = torch.randn(1, 300, 96, generator=g).cuda().bfloat16()
    P = places(300, 1)
    pos = torch.from_numpy(P).cuda()[None]
    X, GY = f64(x)[0], f64(gy)[0]
    if m.shard_major:
        prob = m.problem(1, 300)
        x, gy, pos = (ra.shard_tokens(t.contiguous(), prob) for t in (x, gy, pos))
    x.requires_grad_(True)
    y = m(x, pos)
    y.backward(gy)
    assert ra.check_device_status() == 0, ra.last_error()
    got = {"y": y, "x": x.grad, **{n: p.grad for n, p in m.named_parameters()}}
    if m.shard_major:
        got["y"], got["x"] = (ra.unshard_tokens(got[n].detach().contiguous(), prob) for n in ("y", "x"))
    assert rel(f64(got.pop("y"))[0], reference(m, X, P)) <= TOL
    want = reference(m, X, P, GY)
    assert set(got) == set(want)
    for name in want:  # two more roundings each way: dS, and the gradients of q, k
        a = f64(got[name])[0] if name == "x" else f64(got[name])
        assert rel(a, want[name]) <= 2 * TOL, f"{name}: {rel(a, want[name]):.3e}"


@pytest.mark.parametrize("window", [0, 150])
def test_document_questions_and_answers(window):
    """A document into the cache once, four questions of different lengths behind it in one call, one of
    them in two pieces, then answers token by token in a captured graph: every output is the layer's own on the
    whole sequence."""
    m = layer(window=window, sinks=4 if window else 0)
    page, doc, asks, steps = 16, 640, [30, 5, 1, 77], 6
    g = torch.Generator().manual_seed(8)
    D = torch.randn(doc, 96, generator=g).cuda().bfloat16()
    tails = [torch.randn(n + steps, 96, generator=g).cuda().bfloat16() for n in asks]
    xs = [torch.cat([D, t]) for t in tails]
    P = [np.concatenate([places(doc, 3), 700 + places(n + steps, 10 + i)]) for i, n in enumerate(asks)]
    ps = [torch.from_numpy(p).cuda() for p in P]
    shared_pages = doc // page
    own = [-(-(n + steps) // page) for n in asks]
    pages = shared_pages + sum(own)
    kp = torch.full((pages, page, m.hkv, m.head_dim), float("nan"), device="cuda", dtype=torch.bfloat16)
    vp = torch.full_like(kp, float("nan"))
    width = BIG // (4 * page * m.hkv * m.head_dim * 4) + 1
    table = torch.full((4, width), 1 << 30, dtype=torch.int32)
    at = shared_pages
    for b, n in enumerate(own):
        table[b, :shared_pages] = torch.arange(shared_pages)
        table[b, shared_pages:shared_pages + n] = torch.arange(at, at + n)
        at += n
    cache = ra.make_cache(kp, vp, table.cuda())
    first = ra.make_cache(kp, vp, table[:1].cuda())
    m.prefill(D, first, [0, doc], ps[0][:doc].contiguous())
    ints = lambda *a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    shared = ra.SharedPrefix(ints(0, 4), ints(doc))
    # the last question comes in two pieces
    one = [n if b < 3 else n - 7 for b, n in enumerate(asks)]
    cu = np.concatenate([[0], np.cumsum(one)])
    y = m.extend(torch.cat([t[:n] for t, n in zip(tails, one)]), cache, ints(*(doc + n for n in one)), ints(*cu),
                 torch.cat([p[doc:doc + n] for p, n in zip(ps, one)]), shared)
    ys = [list(y[cu[b]:cu[b + 1]]) for b in range(4)]
    y = m.extend(tails[3][one[3]:asks[3]], cache, ints(*(doc + n for n in asks)), ints(0, 0, 0, 0, 7),
                 ps[3][doc + one[3]:doc + asks[3]], shared)
    ys[3] += list(y)
    lens = ints(*(doc + n for n in asks))
    tok, pos = torch.zeros(4, 96, device="cuda", dtype=torch.bfloat16), torch.zeros(4, 3, device="cuda", dtype=torch.int32)
    ws = torch.empty(max(ra.paged_extend_workspace_bytes(cache, 4, m.hq, shared), ra.paged_workspace_bytes(cache, m.hq)),
                     device="cuda", dtype=torch.uint8)
    m.decode(tok, cache, torch.zeros_like(lens), ws, pos, shared)  # warm-up: every sequence idle
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = m.decode(tok, cache, lens, ws, pos, shared)
    for i in range(steps):
        lens += 1
        for b in range(4):
            tok[b], pos[b] = tails[b][asks[b] + i], ps[b][doc + asks[b] + i]
        graph.replay()
        for b in range(4):
            ys[b].append(y[b].clone())
    assert ra.check_device_status() == 0, ra.last_error()
    for b in range(4):
        got, want = f64(torch.stack(ys[b])), reference(m, f64(xs[b]), P[b])[doc:]
        assert rel(got, want) <= TOL, f"sequence {b}: {rel(got, want):.3e}"
        assert rel(got[-steps:], want[-steps:]) <= TOL


def test_layer_refusals():
    m = layer()
    with pytest.raises(ValueError):
        m(torch.zeros(1, 4, 96, device="cuda", dtype=BF16))  # no positions
    with pytest.raises(ValueError):
        layer(causal=False).extend(None, None, None, None)
    with pytest.raises(ValueError):
        layer(axes=False)(torch.zeros(1, 4, 96, device="cuda", dtype=BF16), torch.zeros(1, 4, 3, device="cuda", dtype=torch.int32))
