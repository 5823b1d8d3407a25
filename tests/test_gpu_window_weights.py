"""Gradients of keys with small weights under a window, against the formulas in float64.

A first token that takes nearly all the weight (what always visible first tokens are for) leaves the
other keys weights of e^-gap / window each; dk and dv of these keys are sums over their own weights,
and are compared on their own. (dq and the first token's dk hang on the first token's dP - delta, a
difference next to 0 that the rounding of `out` inside delta decides, as in the ring's backward.)

Tolerance, relative L2: dS and the result are rounded to bf16, each off by at most half a step of 2^-7
of a number's leading bit, uniformly: 2^-7 / sqrt(12) in the mean square. The row sum dO . out has
`out` rounded likewise; it is one of two like terms of dP - delta, so 2^-7 / sqrt(24). The weights are
halves, 2^-10 / sqrt(12). Together 2^-7 sqrt(1/12 + 1/12 + 1/24 + 1/768) = 0.0036.
"""
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -7 * (1 / 12 + 1 / 12 + 1 / 24 + 1 / 768) ** 0.5


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


def formulas(q, k, v, do, hide, scale):
    """dq, dk, dv of one batch element, [n, heads, dh] float64."""
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    grp = q.shape[1] // k.shape[1]
    for h in range(q.shape[1]):
        x, y, z, w = q[:, h], k[:, h // grp], v[:, h // grp], do[:, h]
        p = torch.softmax((x @ y.T * scale).masked_fill(hide, -float("inf")), -1)
        dp = w @ z.T
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
        dq[:, h] = ds @ y
        dk[:, h // grp] += ds.T @ x
        dv[:, h // grp] += p.T @ w
    return dq, dk, dv


@pytest.mark.parametrize("layout,D", [("basic", 1), ("zigzag", 4), ("stripe", 2)])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("gap", [0, 7, 12, 16, 18])
def test_keys_of_small_weight_keep_their_gradients(layout, D, dh, gap):
    n, hq, hkv, window, sinks = 2048, 2, 1, 1024, 1
    g = torch.Generator().manual_seed(31 + gap)
    q, k, v, do = (torch.randn(1, n, h, dh, generator=g) for h in (hq, hkv, hkv, hq))
    q, k = q * 0.5, k * 0.5
    scale = dh ** -0.5
    q[..., 0], k[..., 0] = 4.0, 0.0
    k[:, 0] = 0.0
    k[:, 0, :, 0] = gap / (4.0 * scale)  # its score is `gap`, the others' are within a few tenths of 0
    q, k, v, do = (t.to(torch.bfloat16).cuda() for t in (q, k, v, do))
    prob = ra.make_problem(dtype=torch.bfloat16, layout=layout, causal=True, D=D, hq=hq, hkv=hkv, head_dim=dh,
                           batch=1, seqlen=n)
    qs, ks, vs, ds = (ra.shard_tokens(t, prob) for t in (q, k, v, do))
    out, lse = ra.window_attn_fwd(qs, ks, vs, prob, window, sinks)
    grads = ra.window_attn_bwd(ds, qs, ks, vs, out, lse, prob, window, sinks)
    assert ra.check_device_status() == 0, ra.last_error()
    i = torch.arange(n, device="cuda")
    hide = ~((i[None] <= i[:, None]) & ((i[None] > i[:, None] - window) | (i[None] < sinks)))
    want = formulas(*(t[0].double() for t in (q, k, v, do)), hide, scale)
    for got, ref, name in zip(grads[1:], want[1:], ("dk", "dv")):
        got = ra.unshard_tokens(got, prob)[0].double()
        rows = slice(1, None)  # without the first token
        off = ((got[rows] - ref[rows]).norm() / ref[rows].norm()).item()
        assert off <= TOL, f"{name}: relative L2 {off:.5f}, allowed {TOL:.5f}"


@pytest.mark.parametrize("window,sinks", [(16, 0), (12, 4), (17, 0), (13, 4), (5, 0), (64, 1)])
@pytest.mark.parametrize("layout,D", [("zigzag", 2), ("stripe", 4)])
def test_gradients_on_both_sides_of_the_row_sums_rule(window, sinks, layout, D):
    """Up to 16 visible keys the row sums come from P and dP, from 17 on from the rounded `out`."""
    n, hq, hkv, dh = 1024, 4, 2, 64
    g = torch.Generator().manual_seed(5)
    q, k, v, do = (torch.randn(1, n, h, dh, generator=g).to(torch.bfloat16).cuda() for h in (hq, hkv, hkv, hq))
    prob = ra.problem_for(q, k, D=D, layout=layout)
    qs, ks, vs, ds = (ra.shard_tokens(t, prob) for t in (q, k, v, do))
    out, lse = ra.window_attn_fwd(qs, ks, vs, prob, window, sinks)
    grads = ra.window_attn_bwd(ds, qs, ks, vs, out, lse, prob, window, sinks)
    again = ra.window_attn_bwd(ds, qs, ks, vs, torch.zeros_like(out), lse, prob, window, sinks)
    assert all(torch.equal(a, b) for a, b in zip(grads, again)) == (window + sinks <= 16)  # `out` is not looked at
    i = torch.arange(n, device="cuda")
    hide = ~((i[None] <= i[:, None]) & ((i[None] > i[:, None] - window) | (i[None] < sinks)))
    want = formulas(*(t[0].double() for t in (q, k, v, do)), hide, dh ** -0.5)
    for got, ref, name in zip(grads, want, ("dq", "dk", "dv")):
        off = ((ra.unshard_tokens(got, prob)[0].double() - ref).norm() / ref.norm()).item()
        assert off <= TOL, f"{name}: relative L2 {off:.5f}, allowed {TOL:.5f}"
