"""Windowed ring attention on the GPU against the dense float64 definition.

Tolerances: bf16 out: the weights are rounded once (2^-8) and the result once, so |err| <= 2^-8
|out| + 1.1 * 2^-8 * sum p |v| elementwise; lse 2^-12 (float32 scores of size < 8 over 128
products). Gradients: dP and delta are float32 sums of dh <= 128 products, each off by at most dh
* 2^-24 * sum |dO v| < 7e-4 here, which times scale and a few keys of size 1 is below 1e-4 an
element (it shows where dP - delta is 0 in exact arithmetic: a query of one key); and four roundings of at most 2^-8 each (weights, dS, the stored out inside
delta, the result), independent: 2^-7 in relative L2. Float32: 1e-5 (out, lse absolute;
gradients relative L2), as for the ring calls.
"""
import numpy as np
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from oracle import heads as H

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


def f64(t):
    return t.detach().double().cpu().numpy()


def check_l2(got, ref, dt, what):
    off, size = np.linalg.norm(got - ref), np.linalg.norm(ref)
    tol = (2.0 ** -7 * size + 1e-4 * ref.size ** 0.5) if dt == BF16 else 1e-5 * size
    assert off <= tol, f"{what}: off by {off:.3e} of {size:.3e}, allowed {tol:.3e}"


def randn(seed, *shape, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


# dtype, layout, D, lens, varlen, hq, hkv, dh, window, sinks
CASES = [
    (BF16, "basic", 1, [700], False, 2, 1, 128, 200, 0),
    (BF16, "basic", 4, [1024, 1024], False, 4, 2, 64, 300, 4),
    (BF16, "basic", 2, [600], False, 4, 4, 128, 1, 0),
    (BF16, "basic", 2, [600], False, 2, 2, 64, 1, 1),
    (BF16, "zigzag", 4, [8 * 130], False, 4, 2, 128, 129, 3),   # chunks of 130 rows: blocks straddle them
    (BF16, "zigzag", 2, [2400], False, 2, 1, 128, 128, 128),
    (BF16, "zigzag", 8, [2048], False, 8, 2, 64, 777, 5),
    (BF16, "stripe", 3, [900], False, 3, 3, 128, 250, 7),
    (BF16, "stripe", 8, [1600], False, 4, 1, 64, 64, 2),
    (BF16, "zigzag", 4, [24, 1200, 0, 8, 512], True, 4, 2, 128, 100, 4),
    (BF16, "basic", 4, [16, 900, 4, 0, 600], True, 4, 4, 128, 40, 30),  # sinks over several shards
    (BF16, "stripe", 2, [10, 700, 2], True, 2, 1, 64, 33, 128),
    (BF16, "zigzag", 40, [400, 800], True, 2, 1, 64, 100, 11),  # more shards than lanes
    (BF16, "basic", 1, [1500], False, 16, 1, 128, 256, 16),
    (BF16, "basic", 2, [256], False, 2, 2, 128, 255, 0),  # all but the farthest pair
    (F32, "stripe", 2, [200], False, 4, 2, 64, 30, 2),
    (F32, "zigzag", 4, [40, 96, 0, 8], True, 2, 1, 33, 9, 3),
    (F32, "basic", 3, [60, 60], False, 3, 3, 1, 20, 128),
    (F32, "stripe", 3, [900], False, 2, 1, 32, 50, 100),
]
IDS = [f"{str(c[0])[6:]}_{c[1]}_D{c[2]}_{max(c[3])}_{c[5]}x{c[6]}_dh{c[7]}_w{c[8]}_s{c[9]}" for c in CASES]


def make(case, seed=1):
    dt, layout, D, lens, varlen, hq, hkv, dh, window, sinks = case
    lead = (sum(lens),) if varlen else (len(lens), lens[0])
    x = [randn(seed + i, *lead, h, dh, dtype=dt) for i, h in enumerate((hq, hkv, hkv, hq))]
    cu = np.concatenate([[0], np.cumsum(lens)]) if varlen else None
    prob = ra.problem_for(x[0], x[1], D=D, layout=layout, causal=True, cu_seqlens=cu)
    return x, prob


def run(x, prob, window, sinks, **kw):
    q, k, v, do = (ra.shard_tokens(t, prob) for t in x)
    out, lse = ra.window_attn_fwd(q, k, v, prob, window, sinks, **kw)
    grads = ra.window_attn_bwd(do, q, k, v, out, lse, prob, window, sinks)
    return out, lse, grads


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_window_forward_and_backward(case):
    dt, layout, D, lens, varlen, hq, hkv, dh, window, sinks = case
    x, prob = make(case)
    out, lse, grads = run(x, prob, window, sinks)
    assert ra.check_device_status() == 0, ra.last_error()
    flat = [f64(t).reshape(-1, *t.shape[-2:]) for t in x]
    nat = [f64(ra.unshard_tokens(t, prob)).reshape(-1, *t.shape[-2:]) for t in (out, *grads)]
    nat_lse = f64(ra.unshard_lse(lse, prob))
    nat_lse = nat_lse if varlen else nat_lse.transpose(1, 0, 2).reshape(hq, -1)
    refs, at = [[] for _ in range(4)], 0
    for n in lens:
        if n == 0:
            continue
        rows = slice(at, at + n)
        at += n
        q, k, v, do = (t[rows] for t in flat)
        ok = H.seen(n, n, window, sinks)
        o, l = H.masked_fwd(q, k, v, ok, dh ** -0.5)
        if dt == BF16:
            spread, _ = H.masked_fwd(q, k, np.abs(v), ok, dh ** -0.5)
            tol = 2.0 ** -8 * np.abs(o) + 1.1 * 2.0 ** -8 * spread
        else:
            tol = 1e-5
        err = np.abs(nat[0][rows] - o)
        assert (err <= tol).all(), f"out: {(~(err <= tol)).sum()} off, worst {err.max()}"
        assert np.abs(nat_lse[:, rows] - l).max() <= (2.0 ** -12 if dt == BF16 else 1e-5)
        for r, g in zip(refs[1:], H.masked_bwd(q, k, v, do, ok, dh ** -0.5)):
            r.append(g)
    for name, got, ref in zip(("dq", "dk", "dv"), nat[1:], refs[1:]):
        ref = np.concatenate(ref)
        assert np.isfinite(got).all(), name
        check_l2(got, ref, dt, name)
        # and where it is easiest to go wrong: the sinks' own rows of every sequence
        first = np.concatenate([np.arange(min(n, max(sinks, 1))) + s for s, n in
                                zip(np.concatenate([[0], np.cumsum(lens)[:-1]]), lens) if n])
        check_l2(got[first], ref[first], dt, name + " of the first rows")


@pytest.mark.parametrize("case", [CASES[1], CASES[9], CASES[15]], ids=["basic", "varlen", "f32"])
def test_window_repeats_bit_for_bit_and_in_graphs(case):
    """Twice, on another stream, captured and replayed with a workspace that holds anything, the
    forward without a workspace: the same bits."""
    window, sinks = case[-2:]
    x, prob = make(case, seed=50)
    out, lse, grads = run(x, prob, window, sinks)
    o2, l2, g2 = run(x, prob, window, sinks)
    assert torch.equal(out, o2) and torch.equal(lse, l2) and all(torch.equal(a, b) for a, b in zip(grads, g2))
    q, k, v, do = (ra.shard_tokens(t, prob) for t in x)
    from context_blockwise_attention_step_gb300 import _abi
    o3, l3 = torch.empty_like(out), torch.empty_like(lse)
    p = lambda t: t.data_ptr()  # noqa: E731
    _abi.check(_abi.lib().ra_window_attn_fwd(prob.ptr, window, sinks, p(q), p(k), p(v), p(o3), p(l3), None, 0,
                                             torch.cuda.current_stream().cuda_stream))
    assert torch.equal(o3, out) and torch.equal(l3, lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o4, l4 = ra.window_attn_fwd(q, k, v, prob, window, sinks, stream=s)
    g4 = ra.window_attn_bwd(do, q, k, v, o4, l4, prob, window, sinks, stream=s)
    s.synchronize()
    assert torch.equal(o4, out) and all(torch.equal(a, b) for a, b in zip(grads, g4))
    ws = [torch.empty(max(256, ra.window_workspace_bytes(prob, window, sinks, i)), device="cuda", dtype=torch.uint8)
          for i in (0, 1)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o5, l5 = ra.window_attn_fwd(q, k, v, prob, window, sinks, workspace=ws[0])
        g5 = ra.window_attn_bwd(do, q, k, v, o5, l5, prob, window, sinks, workspace=ws[1])
    for w in ws:
        w.fill_(0xFF)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o5, out) and torch.equal(l5, lse) and all(torch.equal(a, b) for a, b in zip(grads, g5))


@pytest.mark.parametrize("case", [CASES[4], CASES[11]], ids=["zigzag", "varlen_stripe"])
def test_window_on_the_cuda_cores_in_bf16(case, monkeypatch):
    """The cross-check path (RA_IMPL=simt): no rounding of the weights or of dS there, so it agrees
    with the tensor cores to theirs."""
    window, sinks = case[-2:]
    x, prob = make(case, seed=70)
    out, lse, grads = run(x, prob, window, sinks)
    monkeypatch.setenv("RA_IMPL", "simt")
    o, l, g = run(x, prob, window, sinks)
    assert (lse - l).abs().max() <= 2.0 ** -11
    for a, b, name in zip((out, *grads), (o, *g), ("out", "dq", "dk", "dv")):
        check_l2(f64(a), f64(b), BF16, name)


def test_a_window_over_everything_is_the_ring():
    x, prob = make(CASES[9], seed=60)
    q, k, v, do = (ra.shard_tokens(t, prob) for t in x)
    out, lse = ra.ring_attn_fwd(q, k, v, prob)
    grads = ra.ring_attn_bwd(do, q, k, v, out, lse, prob)
    for window, sinks in ((1200, 0), (2 ** 31 - 1, 128)):
        o, l, g = run(x, prob, window, sinks)
        assert torch.equal(o, out) and torch.equal(l, lse) and all(torch.equal(a, b) for a, b in zip(g, grads))
    o, _, _ = run(x, prob, 1199, 0)  # the last row of the longest sequence loses one key
    assert not torch.equal(o, out)


def test_sinks_alone_carry_the_far_past():
    """A first key that takes all the weight is seen by every query with one sink, and only by
    its window without."""
    n, dh = 640, 64
    q = torch.ones(1, n, 1, dh, device="cuda", dtype=BF16)
    k = torch.zeros_like(q)
    k[0, 0] = 16.0
    v = torch.zeros_like(q)
    v[0, 0] = 1.0
    prob = ra.make_problem(dtype=BF16, layout="basic", causal=True, D=2, hq=1, hkv=1, head_dim=dh, batch=1, seqlen=n)
    with_sink, _ = ra.window_attn_fwd(q, k, v, prob, 100, 1)
    assert (with_sink == 1).all()
    without, lse = ra.window_attn_fwd(q, k, v, prob, 100, 0)
    assert (without[0, :100] == 1).all() and (without[0, 100:] == 0).all()
    assert (lse[0, 0, 100:] - np.log(100)).abs().max() < 1e-5


@pytest.mark.parametrize("layout,D", [("basic", 1), ("zigzag", 4), ("stripe", 2)])
@pytest.mark.parametrize("window,sinks,dh", [(2, 0, 64), (3, 1, 128)])
def test_few_visible_keys_keep_their_gradients(layout, D, window, sinks, dh):
    """dq and dk of a window of two or three keys have two roundings to bf16, of dS and of the
    result: each is off by at most half a step of 2^-7 of a number's leading bit, uniformly, so
    2^-7 / sqrt(12) of the number in the mean square, and both together 2^-7 / sqrt(6) = 0.0032.
    (Row sums dO . O from the bf16 output would put a third and larger one into dS: 0.0038 with two
    keys.)"""
    n, hq, hkv = 768, 4, 2
    q, k, v, do = (randn(91 + i, 1, n, h, dh) for i, h in enumerate((hq, hkv, hkv, hq)))
    prob = ra.make_problem(dtype=BF16, layout=layout, causal=True, D=D, hq=hq, hkv=hkv, head_dim=dh, batch=1, seqlen=n)
    _, _, (dq, dk, _) = run((q, k, v, do), prob, window, sinks)
    dq, dk = (ra.unshard_tokens(t, prob)[0].double() for t in (dq, dk))
    i = torch.arange(n, device="cuda")
    hide = ~((i[None] <= i[:, None]) & ((i[None] > i[:, None] - window) | (i[None] < sinks)))
    want_q, want_k = torch.zeros_like(dq), torch.zeros_like(dk)
    for h in range(hq):
        x, y, z, w = q[0, :, h].double(), k[0, :, h // 2].double(), v[0, :, h // 2].double(), do[0, :, h].double()
        p = torch.softmax((x @ y.T * dh ** -0.5).masked_fill(hide, -1e300), -1)
        dp = w @ z.T
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * dh ** -0.5
        want_q[:, h] = ds @ y
        want_k[:, h // 2] += ds.T @ x
    for got, want in ((dq, want_q), (dk, want_k)):
        assert (got - want).norm() <= 2.0 ** -7 / 6 ** 0.5 * want.norm()
