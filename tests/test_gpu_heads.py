"""Head norms with rotation, the append to a paged cache and the attention over it, on the GPU
against float64.

Tolerances, from the arithmetic (u = 2^-24; `half` = half a step of the stored type, 2^-8 for
bf16 and 2^-24 for f32, relative to the value):
* norm and rotation: the sum of squares takes at most 4 + 5 additions, rsqrt 2 ulp, the weight
  and the rotation 4 roundings, the angle is exact to 2^-25 turn (pi * 2^-24 rad): together below
  2^-20 of the largest element of the head before the rotation.
* its backward: two such heads' products and a second sum: below 2^-18 of the largest term.
* weight gradients: every term to 2^-20, and sums over at most 2^8 terms one after the other,
  then over warps and blocks (below 2^7 more): below 2^-15 of the sum of the terms' magnitudes.
* attention of one token, f32: a score is off by at most dh * u * sum |q k| * scale < 2^-15 here,
  so a weight by 2^-14 relative; bf16 adds the rounding of the weights (2^-8) and of the result.
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


def inv_freq(rd, base=10000.0):
    return base ** (-np.arange(0, rd, 2) / rd)


def positions(layout, D, lens, varlen):
    rows = LY.shard_major_rows(layout, D, lens, varlen=varlen)
    nat = np.concatenate([np.arange(n) for n in lens])
    return nat[np.asarray(rows)]


def close(got, ref, tol, what):
    bad = ~(np.abs(f64(got) - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.abs(f64(got) - ref).max():.3e}"


def amp(x, axis=-1):
    return np.abs(x).max(axis, keepdims=True)


# dtype, layout, D, lens, varlen, hq, hkv, dh, rotary, interleaved
NORM_CASES = [
    (BF16, "zigzag", 4, [64], False, 8, 2, 128, 128, False),
    (BF16, "basic", 2, [6, 6, 6], False, 4, 4, 64, 64, True),
    (BF16, "stripe", 3, [30, 0, 6, 300], True, 6, 2, 128, 64, False),
    (BF16, "zigzag", 2, [4, 8, 0, 0, 400], True, 1, 1, 64, 64, False),
    (BF16, "basic", 1, [1], False, 32, 8, 128, 128, True),
    (F32, "zigzag", 2, [40], False, 4, 1, 128, 128, False),
    (F32, "stripe", 4, [12, 40], True, 2, 2, 96, 48, True),
    (F32, "basic", 1, [17], False, 3, 3, 33, 2, False),
    (F32, "basic", 5, [25, 5], True, 5, 1, 1, None, False),
    (F32, "zigzag", 1, [10], False, 2, 1, 64, 64, True),
    (BF16, "zigzag", 1, [70], False, 5, 5, 128, 16, False),  # rotations of part of the head, in whole
    (BF16, "basic", 2, [12], False, 3, 1, 128, 112, False),  # 16-byte pieces
    (BF16, "basic", 2, [12], False, 3, 1, 64, 22, True),
    (BF16, "basic", 2, [12], False, 3, 1, 64, 22, False),    # and not
    (F32, "stripe", 2, [12], False, 9, 3, 128, 24, False),
    (F32, "stripe", 2, [12], False, 9, 3, 64, 6, True),
    (F32, "zigzag", 2, [40], False, 10, 2, 8, 8, False),      # float32 heads of any multiple of 8
    (F32, "basic", 1, [33], False, 18, 3, 32, 16, False),
    (F32, "basic", 2, [34], False, 6, 3, 24, 10, True),
    (F32, "zigzag", 2, [40], False, 6, 2, 48, 48, False),
    (F32, "stripe", 2, [40], False, 6, 2, 40, 8, False),
    (F32, "zigzag", 2, [40], False, 4, 2, 96, 48, False),
    (F32, "zigzag", 2, [40], False, 4, 2, 80, 80, True),
    (F32, "basic", 2, [40], False, 4, 2, 120, 24, False),
    (F32, "basic", 2, [40], False, 4, 2, 112, None, False),
    (F32, "basic", 2, [40], False, 4, 2, 100, 48, False),
    (F32, "basic", 2, [40], False, 4, 2, 96, 20, False),
]


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: f"{str(c[0])[6:]}_{c[1]}_D{c[2]}_{c[5]}x{c[6]}_dh{c[7]}_r{c[8]}")
@pytest.mark.parametrize("norm,rope", [(True, True), (True, False), (False, True)])
def test_norm_rope_forward_and_backward(case, norm, rope):
    dt, layout, D, lens, varlen, hq, hkv, dh, rd, inter = case
    if rope and rd is None:
        rope, norm = False, True
    n = sum(lens)
    lead = (n,) if varlen else (len(lens), lens[0])
    cu = np.concatenate([[0], np.cumsum(lens)]) if varlen else None
    q, k = randn(1, *lead, hq, dh, dtype=dt, scale=3.0), randn(2, *lead, hkv, dh, dtype=dt, scale=0.2)
    gq, gk = randn(3, *lead, hq, dh, dtype=dt), randn(4, *lead, hkv, dh, dtype=dt)
    wq, wk = randn(5, dh, dtype=dt), randn(6, dh, dtype=dt)
    prob = ra.problem_for(q, k, D=D, layout=layout, cu_seqlens=cu)
    how = dict(q_weight=wq if norm else None, k_weight=wk if norm else None, eps=1e-5,
               rope=ra.make_rope(rd, interleaved=inter) if rope else None)
    q2, k2 = ra.qk_norm_rope_fwd(q, k, prob, **how)
    grads = ra.qk_norm_rope_bwd(gq, gk, q, k, prob, **how)
    z = H.phases(positions(layout, D, lens, varlen), inv_freq(rd)) if rope else None
    for x, y, g, w, dx, dw, h, name in ((q, q2, gq, wq, grads[0], grads[2], hq, "q"),
                                        (k, k2, gk, wk, grads[1], grads[3], hkv, "k")):
        xf, gf, wf = f64(x).reshape(n, h, dh), f64(g).reshape(n, h, dh), f64(w) if norm else None
        ref = H.norm_rope_fwd(xf, wf, z, 1e-5, inter)
        before = amp(H.norm_rope_fwd(xf, wf, None, 1e-5))
        close(y.reshape(n, h, dh), ref, HALF[dt] * np.abs(ref) + 2.0 ** -20 * before * 1.5, name)
        dref, dwref = H.norm_rope_bwd(gf, xf, wf, z, 1e-5, inter)
        if norm:
            r = 1 / np.sqrt((xf * xf).mean(-1, keepdims=True) + 1e-5)
            turned = H.turn(gf, z.conj(), inter) if rope else gf
            hh, nn = turned * wf, xf * r
            size = r * (amp(hh) + amp(nn) * np.abs(hh * nn).mean(-1, keepdims=True))
            close(dw, dwref, 2.0 ** -15 * np.abs(turned * nn).sum((0, 1)) + 1e-30, "dw_" + name)
            assert dw.dtype == F32
        else:
            size = amp(gf) * 1.5
            assert dw is None
        close(dx.reshape(n, h, dh), dref, HALF[dt] * np.abs(dref) + 2.0 ** -18 * size, "d" + name)


def test_norm_rope_views_in_place_streams_and_repeats():
    """A fused projection's views, outputs over the inputs, another stream, captured replays:
    the same bits; the weight gradients repeat bit for bit."""
    n, hq, hkv, dh = 300, 8, 2, 128
    qkv = randn(11, n, hq + 2 * hkv, dh)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    wq, wk = randn(12, dh), randn(13, dh)
    prob = ra.make_problem(dtype=BF16, layout="basic", causal=True, D=2, hq=hq, hkv=hkv, head_dim=dh,
                           cu_seqlens=[0, 200, 300])
    how = dict(q_weight=wq, k_weight=wk, rope=ra.make_rope(dh))
    want = ra.qk_norm_rope_fwd(q.contiguous(), k.contiguous(), prob, **how)
    got = ra.qk_norm_rope_fwd(q, k, prob, **how)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    odd = torch.empty(n * (hq + hkv + 1) * dh + 1, device="cuda", dtype=BF16)[1:].view(n, -1, dh)  # 2-byte aligned
    odd[:, :hq + hkv] = qkv[:, :hq + hkv]
    got = ra.qk_norm_rope_fwd(odd[:, :hq], odd[:, hq:hq + hkv], prob, **how)
    for a, b in zip(got, want):  # another summation order: a step of the type at most
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()
    q1, k1 = q.contiguous(), k.contiguous()
    ra.qk_norm_rope_fwd(q1, k1, prob, q_out=q1, k_out=k1, **how)
    assert torch.equal(q1, want[0]) and torch.equal(k1, want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ra.qk_norm_rope_fwd(q, k, prob, stream=s, **how)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g1, g2 = randn(14, n, hq, dh), randn(15, n, hkv, dh)
    ref = ra.qk_norm_rope_bwd(g1, g2, q, k, prob, **how)
    a1, a2 = g1.clone(), g2.clone()
    again = ra.qk_norm_rope_bwd(a1, a2, q, k, prob, dq=a1, dk=a2, **how)
    assert all(torch.equal(a, b) for a, b in zip(again, ref))
    ws = torch.empty(ra.workspace_bytes(prob, 3), device="cuda", dtype=torch.uint8)
    outs = [torch.zeros_like(x) for x in (g1, g2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = ra.qk_norm_rope_bwd(g1, g2, q, k, prob, dq=outs[0], dk=outs[1], workspace=ws, **how)
    ws.fill_(0xFF)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(res, ref))


def test_far_positions_keep_their_angle():
    """Position 2^17 and beyond: an angle taken as a float product would be off by 2^-7 rad."""
    n = 1 << 19
    q = torch.ones(1, n, 1, 64, device="cuda", dtype=F32)
    prob = ra.make_problem(dtype=F32, layout="basic", causal=True, D=1, hq=1, hkv=1, head_dim=64, batch=1, seqlen=n)
    got, _ = ra.qk_norm_rope_fwd(q, q, prob, rope=ra.make_rope(64))
    at = np.array([0, 1, 131071, 131072, 400003, n - 1])
    ref = H.turn(np.ones((6, 1, 64)), H.phases(at, inv_freq(64)), False)
    close(got[0][torch.from_numpy(at).cuda()], ref, 2.0 ** -20 * 1.5, "far")


# ------------------------------------------------------------------------------ the cache

def make_pages(seed, lens, page, hkv, dh, dt, spare=2, order="nphd", width=0):
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    total = max(1, sum(need)) + spare
    perm = rng.permutation(total)
    width = max([width, 1] + need)
    table = np.full((len(lens), width), -7, dtype=np.int32)  # unused entries are not looked at
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    shape = (total, page, hkv, dh) if order == "nphd" else (total, hkv, page, dh)
    k, v = randn(seed, *shape, dtype=dt), randn(seed + 1, *shape, dtype=dt)
    if order != "nphd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    return k, v, table


APPEND_CASES = [  # dtype, hq, hkv, dh, page, rotary, lens with the new tokens, new tokens (None: one each)
    (BF16, 8, 2, 128, 16, 128, [5, 16, 17, 0, 1], None),
    (BF16, 4, 4, 64, 7, 32, [100, 33, 64], [60, 0, 64]),
    (F32, 3, 1, 50, 1, 50, [4, 9], [4, 1]),
    (F32, 2, 2, 128, 64, None, [70, 64, 3], None),
    (F32, 6, 2, 96, 16, 48, [40, 0, 16], None),
    (F32, 9, 3, 48, 16, 48, [40, 7], [33, 7]),
    (F32, 9, 3, 32, 16, 16, [40, 7], [33, 7]),
    (BF16, 32, 8, 128, 64, 128, [1], None),
]


@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: f"{str(c[0])[6:]}_{c[1]}x{c[2]}_dh{c[3]}_page{c[4]}")
@pytest.mark.parametrize("order", ["nphd", "nhpd"])
def test_append_matches_the_definition_and_touches_nothing_else(case, order):
    dt, hq, hkv, dh, page, rd, lens, new = case
    one = new is None
    new_ = [1 if n else 0 for n in lens] if one else new
    kp, vp, table = make_pages(21, lens, page, hkv, dh, dt, order=order)
    cache = ra.make_cache(kp, vp, torch.from_numpy(table).cuda())
    rows = len(lens) if one else sum(new) + 3  # three rows behind the last sequence
    q, k, v = randn(22, rows, hq, dh, dtype=dt, scale=2.0), randn(23, rows, hkv, dh, dtype=dt), randn(24, rows, hkv, dh, dtype=dt)
    wq, wk = randn(25, dh, dtype=dt), randn(26, dh, dtype=dt)
    k0, v0 = f64(kp), f64(vp)
    q_out = torch.full_like(q, 9.0)
    cu = None if one else torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    ra.check_device_status()
    ra.kv_cache_append(q, k, v, cache, torch.tensor(lens, dtype=torch.int32).cuda(), cu_new=cu, q_weight=wq, k_weight=wk,
                       rope=ra.make_rope(rd) if rd else None, eps=1e-6, q_out=q_out)
    assert ra.check_device_status() == 0, ra.last_error()
    row, kr, vr, qr = 0, k0.copy(), v0.copy(), np.full(q.shape, 9.0)
    ktol = np.zeros_like(kr)
    for b, n in enumerate(lens):
        if one and n == 0:
            qr[row] = 0
            row += 1
        for t in range(n - new_[b], n):
            z = H.phases([t], inv_freq(rd)) if rd else None
            at = table[b, t // page], t % page
            kr[at] = H.norm_rope_fwd(f64(k[row])[None], f64(wk), z, 1e-6)[0]
            ktol[at] = HALF[dt] * np.abs(kr[at]) + 2.0 ** -20 * 1.5 * amp(H.norm_rope_fwd(f64(k[row])[None], f64(wk), None, 1e-6)[0])
            vr[at] = f64(v[row])
            qr[row] = H.norm_rope_fwd(f64(q[row])[None], f64(wq), z, 1e-6)[0]
            row += 1
    np.testing.assert_array_equal(f64(vp), vr)
    close(kp, kr, ktol, "k pages")
    norm_amp = np.sqrt(dh) * np.abs(f64(wq)).max()
    close(q_out, qr, HALF[dt] * np.abs(qr) + 2.0 ** -20 * 1.5 * norm_amp, "q")


def test_append_of_keys_alone_without_norm_copies_bits():
    kp, vp, table = make_pages(31, [40, 3], 16, 2, 128, BF16)
    cache = ra.make_cache(kp, vp, torch.from_numpy(table).cuda())
    kv = randn(32, 1, 43, 4, 128)  # views of one projection
    cu = torch.tensor([0, 40, 43], dtype=torch.int32).cuda()
    assert ra.kv_cache_append(None, kv[:, :, :2], kv[:, :, 2:], cache, torch.tensor([40, 3], dtype=torch.int32).cuda(), cu_new=cu) is None
    for b, (n, r0) in enumerate([(40, 0), (3, 40)]):
        np.testing.assert_array_equal(H.gather(f64(kp), table[b], n), f64(kv[0, r0:r0 + n, :2]))
        np.testing.assert_array_equal(H.gather(f64(vp), table[b], n), f64(kv[0, r0:r0 + n, 2:]))


def test_append_outside_the_cache_is_left_out_and_reported():
    kp, vp, table = make_pages(41, [16, 16, 16, 16], 16, 2, 128, BF16)
    table[1, 0] = kp.shape[0]  # a page that is not there
    cache = ra.make_cache(kp, vp, torch.from_numpy(table).cuda())
    k0 = kp.clone()
    q, k = randn(42, 4, 4, 128), randn(43, 4, 2, 128)
    ra.check_device_status()
    # lengths: fine, a bad page, beyond the table, negative
    q_out = ra.kv_cache_append(q, k, k, cache, torch.tensor([16, 16, 17, -3], dtype=torch.int32).cuda())
    assert ra.check_device_status() == _abi.RA_ERR_CACHE_INDEX
    assert ra.check_device_status() == 0  # reset
    k0[table[0, 0], 15] = k[0]
    assert torch.equal(kp, k0)
    assert torch.equal(q_out[0], q[0]) and (q_out[1:] == 0).all()


# ------------------------------------------------------------------------------ decode

DECODE_CASES = [  # dtype, hq, hkv, dh, page, lens, window, sinks, order
    (BF16, 8, 2, 128, 16, [1, 15, 16, 17, 0, 300, 64, 65], 0, 0, "nphd"),
    (BF16, 32, 8, 128, 64, [700], 0, 0, "nphd"),
    (BF16, 4, 4, 64, 7, [33, 1000, 2], 0, 0, "nhpd"),
    (BF16, 24, 1, 64, 32, [500, 90], 0, 0, "nphd"),  # 24 heads on one K/V head
    (BF16, 16, 1, 128, 16, [129, 0, 4096], 100, 3, "nphd"),
    (BF16, 6, 2, 128, 48, [5, 63, 64, 65, 2000], 64, 5, "nhpd"),
    (BF16, 8, 8, 64, 16, [40, 1, 90], 1, 0, "nphd"),
    (BF16, 8, 8, 64, 16, [40, 9, 90], 8, 200, "nphd"),  # more sinks than keys
    (F32, 3, 1, 50, 5, [1, 77, 0, 200], 0, 0, "nphd"),
    (F32, 8, 1, 128, 64, [1500, 64], 700, 4, "nhpd"),
    (F32, 17, 1, 33, 1, [70], 0, 0, "nphd"),
    (F32, 2, 2, 1, 16, [40], 7, 1, "nphd"),
    (F32, 8, 8, 128, 16, [1, 15, 16, 17, 0, 300, 64, 65], 0, 0, "nphd"),
    (F32, 32, 8, 64, 64, [700, 3], 0, 0, "nphd"),
    (F32, 12, 4, 96, 48, [5, 63, 64, 65, 2000], 64, 5, "nhpd"),
    (F32, 4, 2, 48, 7, [33, 1000, 2], 0, 0, "nhpd"),
    (F32, 16, 2, 32, 16, [40, 1, 90, 0, 500], 30, 2, "nphd"),
    (F32, 5, 1, 100, 16, [129, 0, 4096], 100, 3, "nphd"),
    (F32, 2, 1, 4, 3, [40], 0, 0, "nphd"),
]


def decode_ref(q, kp, vp, table, lens, window, sinks, scale):
    qf, kf, vf = f64(q), f64(kp), f64(vp)
    out, lse, spread = np.zeros(qf.shape), np.full(qf.shape[:2], -np.inf), np.zeros(qf.shape)
    for b, n in enumerate(lens):
        k, v = H.gather(kf, table[b], n), H.gather(vf, table[b], n)
        ok = H.seen(1, n, window, sinks) if n else np.zeros((1, 0), bool)
        o, l = H.masked_fwd(qf[b:b + 1], k, v, ok, scale)
        a, _ = H.masked_fwd(qf[b:b + 1], k, np.abs(v), ok, scale)
        out[b], lse[b], spread[b] = o[0], l[:, 0], a[0]
    return out, lse, spread


def check_decode(out, lse, ref, dt):
    o, l, spread = ref
    tol = HALF[dt] * np.abs(o) + (2.0 ** -8 * 1.1 if dt == BF16 else 2.0 ** -14) * spread
    close(out, o, tol, "out")
    got = f64(lse)
    np.testing.assert_array_equal(np.isneginf(got), np.isneginf(l))
    fin = np.isfinite(l)
    assert (np.abs(got[fin] - l[fin]) <= 2.0 ** -14 + 2.0 ** -22 * np.abs(l[fin])).all()


@pytest.mark.parametrize("case", DECODE_CASES, ids=lambda c: f"{str(c[0])[6:]}_{c[1]}x{c[2]}_dh{c[3]}_page{c[4]}_w{c[6]}")
def test_decode_matches_the_definition(case):
    dt, hq, hkv, dh, page, lens, window, sinks, order = case
    kp, vp, table = make_pages(51, lens, page, hkv, dh, dt, order=order, width=3)
    # what is not visible must not count, whatever it is: rows behind a sequence's end
    for b, n in enumerate(lens):
        if n % page:
            for x in (kp, vp):
                x[int(table[b, n // page]), n % page:] = float("nan")
    cache = ra.make_cache(kp, vp, torch.from_numpy(table).cuda())
    q = randn(52, len(lens), hq, dh, dtype=dt)
    lt = torch.tensor(lens, dtype=torch.int32).cuda()
    out, lse = ra.paged_attn_decode(q, cache, lt, window=window, sinks=sinks)
    assert ra.check_device_status() == 0, ra.last_error()
    check_decode(out, lse, decode_ref(q, kp, vp, table, lens, window, sinks, dh ** -0.5), dt)
    again = ra.paged_attn_decode(q, cache, lt, window=window, sinks=sinks)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_decode_ignores_nan_outside_the_window():
    lens, page = [300], 16
    kp, vp, table = make_pages(61, lens, page, 2, 64, BF16)
    for t in range(4, 300 - 50):
        for x in (kp, vp):
            x[int(table[0, t // page]), t % page] = float("nan")
    q = randn(62, 1, 4, 64)
    cache = ra.make_cache(kp, vp, torch.from_numpy(table).cuda())
    out, lse = ra.paged_attn_decode(q, cache, torch.tensor(lens, dtype=torch.int32).cuda(), window=50, sinks=4)
    check_decode(out, lse, decode_ref(q, torch.nan_to_num(kp), torch.nan_to_num(vp), table, lens, 50, 4, 0.125), BF16)


def test_decode_of_extreme_scores():
    """Scores of several hundred, and keys that are -inf: the running maximum keeps every weight
    finite; a query whose every score is -inf gets 0 and lse -inf, as an idle one does."""
    kp, vp, table = make_pages(71, [600, 70], 16, 1, 128, BF16)
    kp *= 60
    kp[table[1][: 5].tolist()] = -float("inf")
    q = randn(72, 2, 4, 128).abs()
    cache = ra.make_cache(kp, vp, torch.from_numpy(table).cuda())
    out, lse = ra.paged_attn_decode(q, cache, torch.tensor([600, 70], dtype=torch.int32).cuda())
    ref = decode_ref(q[:1], kp, vp, table, [600], 0, 0, 128 ** -0.5)
    # scores near 1000: half an ulp of the scaled score is 2^-15, so weights move by 2^-13
    close(out[:1], ref[0], 2.0 ** -8 * np.abs(ref[0]) + 2.0 ** -7 * ref[2], "out")
    assert (np.abs(f64(lse[:1]) - ref[1]) <= 2.0 ** -11).all()
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()


def test_decode_bad_pages_lengths_and_scale():
    kp, vp, table = make_pages(81, [64, 64], 16, 2, 128, BF16)
    good = torch.from_numpy(table).cuda()
    q = randn(82, 2, 8, 128)
    lens = torch.tensor([64, 64], dtype=torch.int32).cuda()
    want = ra.paged_attn_decode(q, ra.make_cache(kp, vp, good), lens, scale=0.3)
    check_decode(*want, decode_ref(q, kp, vp, table, [64, 64], 0, 0, 0.3), BF16)
    ra.check_device_status()
    for bad in (-1, kp.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = good.clone()
        t[1, 2] = bad
        out, lse = ra.paged_attn_decode(q, ra.make_cache(kp, vp, t), lens, scale=0.3)
        assert ra.check_device_status() == _abi.RA_ERR_CACHE_INDEX
        assert torch.equal(out[0], want[0][0]) and torch.equal(lse[0], want[1][0])  # the other sequence
    for n in (65, 2 ** 31 - 1, -1, -2 ** 31):
        out, lse = ra.paged_attn_decode(q, ra.make_cache(kp, vp, good), torch.tensor([64, n], dtype=torch.int32).cuda(), scale=0.3)
        assert ra.check_device_status() == _abi.RA_ERR_CACHE_INDEX
        assert torch.equal(out[0], want[0][0])
    assert ra.check_device_status() == 0


def test_decode_long_cache_past_32_bit_offsets():
    """A cache of more than 2^31 elements: the pages of the sequence lie at its far end."""
    page, hkv, dh, n = 64, 8, 128, 5000
    total = (1 << 31) // (page * hkv * dh) + 100
    kp = torch.zeros(total, page, hkv, dh, device="cuda", dtype=BF16)
    vp = torch.zeros_like(kp)
    need = -(-n // page)
    kp[-need:], vp[-need:] = randn(91, need, page, hkv, dh), randn(92, need, page, hkv, dh)
    table = torch.arange(total - 1, total - 1 - need, -1, dtype=torch.int32)[None].cuda()
    cache = ra.make_cache(kp, vp, table)
    new = randn(93, 1, hkv, dh)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    ra.kv_cache_append(None, new, new, cache, lens)
    q = randn(94, 1, 32, dh)
    out, lse = ra.paged_attn_decode(q, cache, lens)
    assert torch.equal(kp[total - need, (n - 1) % page], new[0])
    small = torch.arange(need - 1, -1, -1, dtype=torch.int32)[None].numpy()
    ref = decode_ref(q, kp[-need:], vp[-need:], small, [n], 0, 0, dh ** -0.5)
    check_decode(out, lse, ref, BF16)


def test_decode_many_sequences_streams_and_graphs():
    """More sequences than threads of a block, a workspace that two captured graphs share, the
    lengths changed between replays, another stream."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, 700).tolist()
    lens[333] = 5000
    kp, vp, table = make_pages(101, lens, 16, 1, 64, BF16)
    cache = ra.make_cache(kp, vp, torch.from_numpy(table).cuda())
    q = randn(102, 700, 2, 64)
    lt = torch.tensor(lens, dtype=torch.int32).cuda()
    out, lse = ra.paged_attn_decode(q, cache, lt)
    ref = decode_ref(q, kp, vp, table, lens, 0, 0, 0.125)
    check_decode(out, lse, ref, BF16)
    ws = torch.empty(ra.paged_workspace_bytes(cache, 2), device="cuda", dtype=torch.uint8)
    graphs, outs = [], []
    for w in (0, 16):
        g, o, l = torch.cuda.CUDAGraph(), torch.zeros_like(out), torch.zeros_like(lse)
        with torch.cuda.graph(g):
            ra.paged_attn_decode(q, cache, lt, window=w, sinks=2, out=o, lse=l, workspace=ws)
        graphs.append(g)
        outs.append((o, l))
    ws.fill_(0xFF)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], out) and torch.equal(outs[0][1], lse)
    win = ra.paged_attn_decode(q, cache, lt, window=16, sinks=2)
    assert torch.equal(outs[1][0], win[0])
    shorter = [max(0, n - 3) for n in lens]
    lt.copy_(torch.tensor(shorter, dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    check_decode(*outs[0], decode_ref(q, kp, vp, table, shorter, 0, 0, 0.125), BF16)
    s = torch.cuda.Stream()
    o2, l2 = ra.paged_attn_decode(q, cache, lt, stream=s)
    s.synchronize()
    assert torch.equal(o2, outs[0][0]) and torch.equal(l2, outs[0][1])


def test_empty_batches():
    kp, vp, _ = make_pages(111, [4], 16, 2, 64, BF16)
    cache = ra.make_cache(kp, vp, torch.zeros(0, 4, dtype=torch.int32).cuda())
    q = randn(112, 0, 4, 64)
    none = torch.zeros(0, dtype=torch.int32).cuda()
    out, lse = ra.paged_attn_decode(q, cache, none)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert ra.kv_cache_append(q, q[:, :2], q[:, :2], cache, none).shape == (0, 4, 64)
    prob = ra.make_problem(dtype=BF16, layout="zigzag", causal=True, D=2, hq=4, hkv=2, head_dim=64, cu_seqlens=[0, 0, 0])
    w = randn(113, 64)
    how = dict(q_weight=w, k_weight=w, rope=ra.make_rope(64))
    assert ra.qk_norm_rope_fwd(q, q[:, :2], prob, **how)[0].shape == (0, 4, 64)
    grads = ra.qk_norm_rope_bwd(q, q[:, :2].contiguous(), q, q[:, :2], prob, **how)
    assert (grads[2] == 0).all() and (grads[3] == 0).all()


def test_rows_past_32_bit_offsets():
    """Rows 2^30 elements apart: the last of four starts past 2^31."""
    wide = torch.empty(4, 1 << 30, device="cuda", dtype=BF16)
    q, k = wide[:, :512].view(4, 4, 128), wide[:, 512:768].view(4, 2, 128)
    q.copy_(randn(121, 4, 4, 128))
    k.copy_(randn(122, 4, 2, 128))
    prob = ra.make_problem(dtype=BF16, layout="basic", causal=True, D=1, hq=4, hkv=2, head_dim=128, cu_seqlens=[0, 4])
    w = randn(123, 128)
    how = dict(q_weight=w, k_weight=w, rope=ra.make_rope(128))
    for a, b in zip(ra.qk_norm_rope_fwd(q, k, prob, **how), ra.qk_norm_rope_fwd(q.clone(), k.clone(), prob, **how)):
        assert torch.equal(a, b)
    g1, g2 = randn(124, 4, 4, 128), randn(125, 4, 2, 128)
    for a, b in zip(ra.qk_norm_rope_bwd(g1, g2, q, k, prob, **how), ra.qk_norm_rope_bwd(g1, g2, q.clone(), k.clone(), prob, **how)):
        assert torch.equal(a, b)
    kp, vp, table = make_pages(126, [4], 16, 2, 128, BF16)
    cache = ra.make_cache(kp, vp, torch.from_numpy(table).cuda())
    cu = torch.tensor([0, 4], dtype=torch.int32).cuda()
    ra.kv_cache_append(q, k, k, cache, cu[1:], cu_new=cu)
    assert torch.equal(vp[int(table[0, 0]), :4], k)


def test_calls_at_once_on_two_streams():
    """Decodes and windowed attention side by side, each with its own outputs and workspace."""
    lens = [3000, 5, 700]
    kp, vp, table = make_pages(131, lens, 16, 2, 128, BF16)
    cache = ra.make_cache(kp, vp, torch.from_numpy(table).cuda())
    q = randn(132, 3, 8, 128)
    lt = torch.tensor(lens, dtype=torch.int32).cuda()
    x = [randn(133 + i, 1, 1024, h, 128) for i, h in enumerate((8, 2, 2))]
    prob = ra.make_problem(dtype=BF16, layout="zigzag", causal=True, D=2, hq=8, hkv=2, head_dim=128, batch=1, seqlen=1024)
    want = ra.paged_attn_decode(q, cache, lt), ra.window_attn_fwd(*x, prob, 100, 3)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(20):
        got.append((ra.paged_attn_decode(q, cache, lt, stream=streams[0]), ra.paged_attn_decode(q, cache, lt, stream=streams[1]),
                    ra.window_attn_fwd(*x, prob, 100, 3, stream=streams[2])))
    torch.cuda.synchronize()
    for a, b, c in got:
        for u, v in zip((*a, *b, *c), (*want[0], *want[0], *want[1])):
            assert torch.equal(u, v)
    assert ra.check_device_status() == 0
