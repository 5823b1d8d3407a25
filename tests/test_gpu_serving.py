"""The operators together: a layer with head norms, rotation, window and sinks trained over ring
shards, and the same layer serving the same tokens from a paged cache.

A token's output is the same function of the same inputs on both ways; they differ by roundings to
bf16 (2^-8 relative each): the projected and the normed q and k, the weights and the attention's
output, and the output projection's result: six in all, independent, so 2^-8 * sqrt(6) < 2^-6.5 in
relative L2 against float64, and twice that between the two ways.
"""
import numpy as np
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from oracle import heads as H

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -6.5


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


def f64(t):
    return t.detach().double().cpu().numpy()


def rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def layer(dh=64, hq=4, hkv=2, window=0, sinks=0, rope=True, norm=True, **kw):
    m = ra.RingSelfAttention(96, hq, hkv, dh, device="cuda", seed=5, qk_norm=norm, window=window, sinks=sinks,
                             rope=ra.make_rope(dh) if rope else None, **{"D": 2, "layout": "zigzag", **kw})
    if norm:
        with torch.no_grad():
            g = torch.Generator().manual_seed(6)
            for w in (m.q_norm, m.k_norm):
                w.copy_(1 + 0.3 * torch.randn(dh, generator=g))
    return m


def reference(m, X, GY=None):
    """y, or with GY the gradients of x and of every parameter, float64, of one sequence X [n, hidden]."""
    W = {n: f64(p) for n, p in m.named_parameters()}
    n = X.shape[0]
    inv = 10000.0 ** (-np.arange(0, m.head_dim, 2) / m.head_dim)
    z = H.phases(np.arange(n), inv) if m.rope is not None else None
    q0, k0 = (X @ W["wq"].T).reshape(n, m.hq, -1), (X @ W["wk"].T).reshape(n, m.hkv, -1)
    v = (X @ W["wv"].T).reshape(n, m.hkv, -1)
    q, k = (H.norm_rope_fwd(t, W.get(w), z, m.eps) for t, w in ((q0, "q_norm"), (k0, "k_norm")))
    ok, scale = H.seen(n, n, m.window, m.sinks), m.head_dim ** -0.5
    out, _ = H.masked_fwd(q, k, v, ok, scale)
    if GY is None:
        return out.reshape(n, -1) @ W["wo"].T
    dq, dk, dv = H.masked_bwd(q, k, v, (GY @ W["wo"]).reshape(out.shape), ok, scale)
    dq, dqn = H.norm_rope_bwd(dq, q0, W.get("q_norm"), z, m.eps)
    dk, dkn = H.norm_rope_bwd(dk, k0, W.get("k_norm"), z, m.eps)
    flat = lambda t: t.reshape(n, -1)  # noqa: E731
    g = {"x": flat(dq) @ W["wq"] + flat(dk) @ W["wk"] + flat(dv) @ W["wv"], "wq": flat(dq).T @ X,
         "wk": flat(dk).T @ X, "wv": flat(dv).T @ X, "wo": GY.T @ flat(out)}
    if dqn is not None:
        g.update(q_norm=dqn, k_norm=dkn)
    return g


@pytest.mark.parametrize("kw", [dict(), dict(window=50, sinks=3), dict(window=40, norm=False, layout="stripe"),
                                dict(rope=False, dh=128, D=1, layout="basic")], ids=str)
def test_layer_output_and_gradients(kw):
    m = layer(**kw)
    g = torch.Generator().manual_seed(7)
    x = torch.randn(1, 300, 96, generator=g).cuda().bfloat16().requires_grad_(True)
    gy = torch.randn(1, 300, 96, generator=g).cuda().bfloat16()
    y = m(x)
    y.backward(gy)
    assert ra.check_device_status() == 0, ra.last_error()
    X, GY = f64(x)[0], f64(gy)[0]
    assert rel(f64(y)[0], reference(m, X)) <= TOL
    want = reference(m, X, GY)
    got = {"x": f64(x.grad)[0], **{n: f64(p.grad) for n, p in m.named_parameters()}}
    assert set(got) == set(want)
    for name in want:
        # two more roundings each way: dS, and the gradients of q, k
        assert rel(got[name], want[name]) <= 2 * TOL, f"{name}: {rel(got[name], want[name]):.3e}"


@pytest.mark.parametrize("kw", [dict(), dict(window=30, sinks=4), dict(dh=128, norm=False, window=17)], ids=str)
def test_prefill_and_decode_are_the_layer(kw):
    """Three sequences, one idle: prompts into the cache, then token by token in a captured graph,
    against the whole sequences at once."""
    m = layer(**kw)
    prompts, steps, page = [70, 33, 0], 20, 16
    g = torch.Generator().manual_seed(8)
    xs = [torch.randn(n + (steps if n else 0), 96, generator=g).cuda().bfloat16() for n in prompts]
    pages = sum(-(-(n + steps) // page) for n in prompts)
    kp = torch.full((pages, page, m.hkv, m.head_dim), float("nan"), device="cuda", dtype=torch.bfloat16)
    vp = torch.full_like(kp, float("nan"))
    table = torch.zeros(3, 6, dtype=torch.int32)
    at = iter(torch.randperm(pages, generator=g).tolist())
    for b, n in enumerate(prompts):
        for i in range(-(-(n + steps) // page)):
            table[b, i] = next(at)
    cache = ra.make_cache(kp, vp, table.cuda())
    cu = np.concatenate([[0], np.cumsum(prompts)])
    ys = [list(t) for t in torch.split(m.prefill(torch.cat([x[:n] for x, n in zip(xs, prompts)]), cache, cu), prompts)]
    lens = torch.tensor(prompts, dtype=torch.int32).cuda()
    tok = torch.zeros(3, 96, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(ra.paged_workspace_bytes(cache, m.hq), device="cuda", dtype=torch.uint8)
    m.decode(tok, cache, torch.zeros_like(lens), workspace=ws)  # warm-up: every sequence idle
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = m.decode(tok, cache, lens, workspace=ws)
    for i in range(steps):
        lens += torch.tensor([1, 1, 0], dtype=torch.int32).cuda()
        for b in (0, 1):
            tok[b] = xs[b][prompts[b] + i]
        graph.replay()
        assert (y[2] == 0).all()
        for b in (0, 1):
            ys[b].append(y[b].clone())
    assert ra.check_device_status() == 0, ra.last_error()
    for b in (0, 1):
        got, want = f64(torch.stack(ys[b])), reference(m, f64(xs[b]))
        assert rel(got, want) <= TOL, f"sequence {b}: {rel(got, want):.3e}"
        assert rel(got[-steps:], want[-steps:]) <= TOL
    m2 = layer(**{**kw, "D": 1, "layout": "basic"})  # the training form, one sequence at a time
    for b in (0, 1):
        assert rel(f64(torch.stack(ys[b])), f64(m2(xs[b][None]))[0]) <= 2 * TOL


def test_training_step_in_a_graph():
    """Forward and backward captured; replayed on new inputs they give the eager gradients."""
    m = layer(window=30, sinks=2)
    x = torch.randn(1, 128, 96, device="cuda").bfloat16()
    gy = torch.randn(1, 128, 96, device="cuda").bfloat16()
    params = list(m.parameters())
    step = lambda: torch.autograd.grad(m(x), params, gy)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step()
    x.copy_(torch.randn(1, 128, 96, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(grads, step()):
        assert torch.equal(a, b)


def test_layer_refusals():
    with pytest.raises(ValueError):
        layer(sinks=3)
    m = layer(causal=False)
    with pytest.raises(ValueError):
        m.decode(None, None, None)
    with pytest.raises(ValueError):
        ra.ring_attention(None, None, None, None, window=0, sinks=1)
