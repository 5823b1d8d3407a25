"""Pins of oracle/heads.py to things other than itself (CPU only): finite differences, scalar
loops, and the plain attention oracle."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import heads as H


def _rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_scalar_loop_and_depends_on_distance_only(interleaved):
    rng = _rng(1)
    x, inv = rng.standard_normal((5, 2, 12)), [0.7, 0.2, 0.01]  # rotates 6 of 12 elements
    pos = np.array([0, 3, 9, 100000, 1 << 30])
    y = H.turn(x, H.phases(pos, inv), interleaved)
    for t in range(5):
        for h in range(2):
            for i, f in enumerate(inv):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 3)
                c, s = np.cos(pos[t] * f), np.sin(pos[t] * f)
                assert abs(y[t, h, a] - (x[t, h, a] * c - x[t, h, b] * s)) < 1e-12
                assert abs(y[t, h, b] - (x[t, h, b] * c + x[t, h, a] * s)) < 1e-12
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
    q, k = rng.standard_normal((1, 1, 6)), rng.standard_normal((1, 1, 6))
    dots = [(H.turn(q, H.phases([m + 40], inv), interleaved) *
             H.turn(k, H.phases([m], inv), interleaved)).sum() for m in (0, 17, 900)]
    np.testing.assert_allclose(dots, dots[0], rtol=0, atol=1e-12)


@pytest.mark.parametrize("norm,rope", [(True, True), (True, False), (False, True)])
def test_norm_rope_gradient_by_differences(norm, rope):
    rng = _rng(2)
    x, dy = rng.standard_normal((3, 2, 8)), rng.standard_normal((3, 2, 8))
    w = 1 + 0.3 * rng.standard_normal(8) if norm else None
    z = H.phases([0, 5, 77], [0.9, 0.1]) if rope else None
    dx, dw = H.norm_rope_bwd(dy, x, w, z, 1e-3)
    f = lambda x, w: (H.norm_rope_fwd(x, w, z, 1e-3) * dy).sum()  # noqa: E731
    e = 1e-6
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = e
        assert abs((f(x + d, w) - f(x - d, w)) / (2 * e) - dx[i]) < 1e-7
    for i in range(8 if norm else 0):
        d = np.zeros(8)
        d[i] = e
        assert abs((f(x, w + d) - f(x, w - d)) / (2 * e) - dw[i]) < 1e-7


def test_masked_attention_is_plain_attention_under_the_causal_mask():
    rng = _rng(3)
    q, k, v, do = (rng.standard_normal((9, h, 4)) for h in (4, 2, 2, 4))
    cu = np.array([0, 9])
    ok, scale = H.seen(9, 9, 0, 0), A.default_scale(4)
    out, lse = H.masked_fwd(q, k, v, ok, scale)
    ref, lref = A.attention_fwd(q, k, v, cu, True)
    np.testing.assert_allclose(out, ref, atol=1e-13)
    np.testing.assert_allclose(lse, lref, atol=1e-13)
    for a, b in zip(H.masked_bwd(q, k, v, do, ok, scale), A.attention_bwd(q, k, v, do, cu, True)):
        np.testing.assert_allclose(a, b, atol=1e-12)
    full = H.seen(9, 9, 9, 0)
    np.testing.assert_array_equal(full, ok)


def test_window_mask_by_loops_and_gradient_by_differences():
    for n, w, s in [(7, 1, 0), (7, 3, 2), (7, 3, 9), (5, 5, 1), (6, 2, 1)]:
        ok = H.seen(n, n, w, s)
        for p in range(n):
            for j in range(n):
                assert ok[p, j] == (j <= p and (p - j < w or j < s))
    rng = _rng(4)
    q, k, v, do = (rng.standard_normal((6, h, 3)) for h in (2, 1, 1, 2))
    ok = H.seen(6, 6, 2, 1)
    grads = H.masked_bwd(q, k, v, do, ok, 0.6)
    e = 1e-6
    for name, x, g in zip("qkv", (q, k, v), grads):
        for i in np.ndindex(x.shape):
            d = np.zeros_like(x)
            d[i] = e
            f = [(H.masked_fwd(*[t + (sgn * d if n == name else 0) for n, t in zip("qkv", (q, k, v))],
                               ok, 0.6)[0] * do).sum() for sgn in (1, -1)]
            assert abs((f[0] - f[1]) / (2 * e) - g[i]) < 1e-7


def test_gather_and_empty_rows():
    pages = _rng(5).standard_normal((4, 3, 2, 5))
    got = H.gather(pages, [2, 0, 3], 7)
    assert got.shape == (7, 2, 5)
    for t, (p, s) in enumerate([(2, 0), (2, 1), (2, 2), (0, 0), (0, 1), (0, 2), (3, 0)]):
        np.testing.assert_array_equal(got[t], pages[p, s])
    out, lse = H.masked_fwd(np.ones((1, 2, 5)), np.zeros((0, 2, 5)), np.zeros((0, 2, 5)),
                            np.zeros((1, 0), bool), 1.0)
    assert (out == 0).all() and np.isneginf(lse).all()
