"""Head norms and the append to a paged cache with positions on several axes, on the GPU against float64,
and the layer that uses them.

Tolerances as for positions on one axis, the arithmetic being the same (u = 2^-24; `half` = half a step
of the stored type): a norm with its rotation is off by less than 2^-20 of the head's largest element
before the rotation, its backward by 2^-18 of the largest term, a weight gradient by 2^-15 of the sum
of the terms' magnitudes; each with its rounding to the stored type.
"""
import numpy as np
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from context_blockwise_attention_step_gb300 import _abi
from oracle import heads as H
from oracle import layouts as LY

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def close(got, ref, tol, what):
    bad = ~(np.abs(f64(got) - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.abs(f64(got) - ref).max():.3e}"


def amp(x, axis=-1):
    return np.abs(x).max(axis, keepdims=True)


def inv_freq(rd, base=10000.0):
    return base ** (-np.arange(0, rd, 2) / rd)


def positions_of(seed, *lead, axes=3, lo=-50, hi=70000):
    """Any positions: far ones, negative ones, equal ones."""
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(lo, hi, (*lead, axes), generator=g, dtype=torch.int32)
    p.view(-1, axes)[::5] = 7
    return p


CASES = [
    # dtype, layout, D, lens, varlen, hq, hkv, dh, rotary, interleaved, axis of every pair
    (BF16, "zigzag", 4, [64], False, 8, 2, 128, 128, False, ra.axis_sections([16, 24, 24])),
    (BF16, "basic", 2, [6, 6, 6], False, 4, 4, 64, 64, True, ra.axis_sections([12, 10, 10], cyclic=True)),
    (BF16, "stripe", 3, [30, 0, 6, 300], True, 6, 2, 128, 64, False, ra.axis_sections([16, 16])),
    (BF16, "basic", 1, [1], False, 32, 8, 128, 128, True, [7] * 64),
    (BF16, "basic", 2, [12], False, 3, 1, 64, 22, False, ra.axis_sections([4, 4, 3])),  # not in 16-byte pieces
    (BF16, "zigzag", 1, [70], False, 5, 5, 128, 112, False, ra.axis_sections([20, 18, 18], cyclic=True)),
    (F32, "stripe", 4, [12, 40], True, 2, 2, 96, 48, True, ra.axis_sections([12, 12])),
    (F32, "basic", 1, [17], False, 3, 3, 33, 2, False, [0]),
    (F32, "zigzag", 2, [40], False, 10, 2, 8, 8, False, [0, 1, 2, 3]),
    (F32, "basic", 2, [40], False, 4, 2, 100, 48, False, ra.axis_sections([8, 8, 8])),
    (F32, "zigzag", 2, [40], False, 4, 1, 128, 128, False, ra.axis_sections([8] * 8)),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0])[6:]}_{c[1]}_D{c[2]}_{c[5]}x{c[6]}_dh{c[7]}_r{c[8]}")
@pytest.mark.parametrize("norm", [True, False])
def test_norm_and_rotation(case, norm):
    dt, layout, D, lens, varlen, hq, hkv, dh, rd, inter, axis = case
    n, axes = sum(lens), max(axis) + 1
    lead = (n,) if varlen else (len(lens), lens[0])
    cu = np.concatenate([[0], np.cumsum(lens)]) if varlen else None
    q, k = randn(1, *lead, hq, dh, dtype=dt, scale=3.0), randn(2, *lead, hkv, dh, dtype=dt, scale=0.2)
    gq, gk = randn(3, *lead, hq, dh, dtype=dt), randn(4, *lead, hkv, dh, dtype=dt)
    wq, wk = randn(5, dh, dtype=dt), randn(6, dh, dtype=dt)
    prob = ra.problem_for(q, k, D=D, layout=layout, cu_seqlens=cu)
    natural = positions_of(7, *lead, axes=axes)
    rows = np.asarray(LY.shard_major_rows(layout, D, lens, varlen=varlen))
    pos = ra.shard_tokens(natural.cuda(), prob)  # the library's own way into shard-major order
    np.testing.assert_array_equal(pos.cpu().numpy().reshape(n, axes), natural.numpy().reshape(n, axes)[rows])
    how = dict(q_weight=wq if norm else None, k_weight=wk if norm else None, eps=1e-5, positions=pos,
               rope=ra.make_axis_rope(rd, axis, interleaved=inter))
    q2, k2 = ra.qk_norm_rope_fwd(q, k, prob, **how)
    grads = ra.qk_norm_rope_bwd(gq, gk, q, k, prob, **how)
    z = H.axis_phases(pos.cpu().numpy().reshape(n, axes), axis, inv_freq(rd))
    for x, y, g, w, dx, dw, h, name in ((q, q2, gq, wq, grads[0], grads[2], hq, "q"),
                                        (k, k2, gk, wk, grads[1], grads[3], hkv, "k")):
        xf, gf, wf = f64(x).reshape(n, h, dh), f64(g).reshape(n, h, dh), f64(w) if norm else None
        ref = H.norm_rope_fwd(xf, wf, z, 1e-5, inter)
        before = amp(H.norm_rope_fwd(xf, wf, None, 1e-5))
        close(y.reshape(n, h, dh), ref, HALF[dt] * np.abs(ref) + 2.0 ** -20 * before * 1.5, name)
        dref, dwref = H.norm_rope_bwd(gf, xf, wf, z, 1e-5, inter)
        if norm:
            r = 1 / np.sqrt((xf * xf).mean(-1, keepdims=True) + 1e-5)
            turned = H.turn(gf, z.conj(), inter)
            hh, nn = turned * wf, xf * r
            size = r * (amp(hh) + amp(nn) * np.abs(hh * nn).mean(-1, keepdims=True))
            close(dw, dwref, 2.0 ** -15 * np.abs(turned * nn).sum((0, 1)) + 1e-30, "dw_" + name)
        else:
            size = amp(gf) * 1.5
            assert dw is None
        close(dx.reshape(n, h, dh), dref, HALF[dt] * np.abs(dref) + 2.0 ** -18 * size, "d" + name)
    again = ra.qk_norm_rope_bwd(gq, gk, q, k, prob, **how)
    assert all(a is b or torch.equal(a, b) for a, b in zip(grads, again))


def test_equal_positions_are_the_rotation_by_place():
    """Positions that are a token's place on every axis: bit for bit the calls without axes, for a
    strided view of positions, in place, on another stream and replayed from a graph."""
    n, hq, hkv, dh = 300, 8, 2, 128
    q, k = randn(11, n, hq, dh), randn(12, n, hkv, dh)
    wq, wk = randn(13, dh), randn(14, dh)
    prob = ra.make_problem(dtype=BF16, layout="stripe", causal=True, D=2, hq=hq, hkv=hkv, head_dim=dh,
                           cu_seqlens=[0, 200, 300])
    want = ra.qk_norm_rope_fwd(q, k, prob, q_weight=wq, k_weight=wk, rope=ra.make_rope(dh))
    place = torch.cat([torch.arange(200), torch.arange(100)]).int().cuda()
    pos = ra.shard_tokens(place[:, None].expand(n, 3).contiguous(), prob)
    wide = torch.full((n, 7), -1, device="cuda", dtype=torch.int32)
    wide[:, 2:5] = pos
    how = dict(q_weight=wq, k_weight=wk, rope=ra.make_axis_rope(dh, ra.axis_sections([16, 24, 24])))
    for p in (pos, wide[:, 2:5]):
        got = ra.qk_norm_rope_fwd(q, k, prob, positions=p, **how)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ra.qk_norm_rope_fwd(q, k, prob, positions=pos, stream=s, **how)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    q1, k1 = torch.empty_like(q), torch.empty_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.qk_norm_rope_fwd(q, k, prob, positions=pos, q_out=q1, k_out=k1, **how)
    keep = pos.clone()
    pos.zero_()
    graph.replay()  # reads the positions of the replay
    pos.copy_(keep)
    flat = ra.qk_norm_rope_fwd(q, k, prob, positions=torch.zeros_like(pos), **how)
    assert torch.equal(q1, flat[0])
    graph.replay()
    assert torch.equal(q1, want[0]) and torch.equal(k1, want[1])
    ra.qk_norm_rope_fwd(q, k, prob, positions=pos, q_out=q, k_out=k, **how)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_the_largest_positions_keep_their_angle():
    at = np.array([[2 ** 31 - 1, 0], [-2 ** 31, 5], [2 ** 30 + 1, -1], [131072, 2 ** 31 - 1]], np.int64)
    axis = ra.axis_sections([16, 16])
    q = torch.ones(4, 1, 64, device="cuda", dtype=F32)
    prob = ra.make_problem(dtype=F32, layout="basic", causal=True, D=1, hq=1, hkv=1, head_dim=64, cu_seqlens=[0, 4])
    # frequencies whose turns are whole multiples of 2^-20: the angle is exact in integers
    turns = np.arange(1, 33) * 37
    got, _ = ra.qk_norm_rope_fwd(q, q, prob, rope=ra.make_axis_rope(64, axis, inv_freq=turns * (2 * np.pi / 2 ** 20)),
                                 positions=torch.from_numpy(at).int().cuda())
    part = np.stack([at[:, a] * t % 2 ** 20 for a, t in zip(axis, turns.tolist())], -1)
    ref = H.turn(np.ones((4, 1, 64)), np.exp(2j * np.pi * part / 2 ** 20), False)
    # 2^-26 of a turn, and what the frequency is off by as a double (2^-53 relative of 2^-10 turns) times 2^31
    close(got, ref, 1.5 * (2.0 ** -20 + 2 * np.pi * 2.0 ** -30), "far")


@pytest.mark.parametrize("dt,dh,page", [(BF16, 128, 16), (BF16, 64, 7), (F32, 96, 16), (F32, 33, 5)], ids=str)
@pytest.mark.parametrize("one", [True, False])
def test_append(dt, dh, page, one):
    hq, hkv = 6, 2
    lens = [5, 16, 17, 0, 1] if one else [40, 3, 33]
    new = [1, 1, 1, 0, 1] if one else [33, 3, 0]
    rd = dh // 2 * 2
    axis = [i % 3 for i in range(rd // 2)]
    rows = len(lens) if one else sum(new) + 2  # two rows behind the last sequence
    q, k, v = randn(22, rows, hq, dh, dtype=dt, scale=2.0), randn(23, rows, hkv, dh, dtype=dt), randn(24, rows, hkv, dh, dtype=dt)
    wq, wk = randn(25, dh, dtype=dt), randn(26, dh, dtype=dt)
    pos = positions_of(27, rows).cuda()
    need = [-(-n // page) for n in lens]
    table = np.full((len(lens), max(need)), -7, np.int32)
    perm, at = np.random.default_rng(28).permutation(sum(need) + 2), 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    kp = torch.full((sum(need) + 2, page, hkv, dh), 5.0, device="cuda", dtype=dt)
    vp = kp.clone()
    cache = ra.make_cache(kp, vp, torch.from_numpy(table).cuda())
    cu = None if one else torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    q_out = torch.full_like(q, 9.0)
    ra.check_device_status()
    ra.kv_cache_append(q, k, v, cache, torch.tensor(lens, dtype=torch.int32).cuda(), cu_new=cu, q_weight=wq, k_weight=wk,
                       rope=ra.make_axis_rope(rd, axis), eps=1e-6, q_out=q_out, positions=pos)
    assert ra.check_device_status() == 0, ra.last_error()
    z = H.axis_phases(pos.cpu().numpy(), axis, inv_freq(rd))
    kref, vref, ktol = np.full(kp.shape, 5.0), np.full(kp.shape, 5.0), np.zeros(kp.shape)
    qref = np.full(q.shape, 9.0)
    row = 0
    for b, n in enumerate(lens):
        if one and n == 0:
            qref[row] = 0
            row += 1
        for t in range(n - new[b], n):
            to, zr = (table[b, t // page], t % page), z[row:row + 1]
            kref[to] = H.norm_rope_fwd(f64(k[row])[None], f64(wk), zr, 1e-6)[0]
            ktol[to] = HALF[dt] * np.abs(kref[to]) + 2.0 ** -20 * 1.5 * amp(H.norm_rope_fwd(f64(k[row])[None], f64(wk), None, 1e-6)[0])
            vref[to] = f64(v[row])
            qref[row] = H.norm_rope_fwd(f64(q[row])[None], f64(wq), zr, 1e-6)[0]
            row += 1
    np.testing.assert_array_equal(f64(vp), vref)
    close(kp, kref, ktol, "k pages")
    close(q_out, qref, HALF[dt] * np.abs(qref) + 2.0 ** -20 * 1.5 * np.sqrt(dh) * np.abs(f64(wq)).max(), "q")


def test_gradient_of_the_differentiable_call():
    """Autograd's gradients are the direct calls', with and without a norm; positions have none."""
    n, hq, hkv, dh = 40, 4, 2, 64
    prob = ra.make_problem(dtype=BF16, layout="basic", causal=True, D=2, hq=hq, hkv=hkv, head_dim=dh, batch=1, seqlen=n)
    pos, rope = positions_of(31, 1, n).cuda(), ra.make_axis_rope(dh, ra.axis_sections([8, 12, 12]))
    gq, gk = randn(32, 1, n, hq, dh), randn(33, 1, n, hkv, dh)
    for norm in (True, False):
        q, k = randn(34, 1, n, hq, dh).requires_grad_(True), randn(35, 1, n, hkv, dh).requires_grad_(True)
        wq, wk = (randn(36, dh).requires_grad_(True), randn(37, dh).requires_grad_(True)) if norm else (None, None)
        y = ra.qk_norm_rope(q, k, prob, wq, wk, rope, 1e-6, pos)
        inputs = [q, k] + ([wq, wk] if norm else [])
        got = torch.autograd.grad(y, inputs, (gq, gk))
        want = ra.qk_norm_rope_bwd(gq, gk, q.detach(), k.detach(), prob, wq, wk, rope, 1e-6, positions=pos)
        for a, b in zip(got, want):
            assert torch.equal(a, b.to(a.dtype))
