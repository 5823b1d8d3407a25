"""The weights of the bf16 decode attention: the result's own rounding is the only one that shows.

A score is a float32 sum of dh <= 128 exact products, off by at most dh * 2^-24 * sum |q k| * scale <
2^-14 here; P is held to 2^-16 (two bf16 numbers, each off by at most 2^-8 of what it rounds); the
sums over the keys are float32, at most 2^10 additions one after the other on a warp's way: 2^-14,
for the numerator and for the denominator. Together below 2^-12 of sum p |v|, and 2^-8 of `out` for
its rounding. (One bf16 number for P would put up to 2^-8 of sum p |v| there.)
"""
import numpy as np
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from oracle import heads as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


def make(seed, lens, hq, hkv, dh, page=16):
    g = torch.Generator().manual_seed(seed)
    width = max((n + page - 1) // page for n in lens) + 1
    n_pages = len(lens) * width
    kp, vp = (torch.randn(n_pages, page, hkv, dh, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    table = torch.randperm(n_pages, generator=g).to(torch.int32).view(len(lens), width)
    q = torch.randn(len(lens), hq, dh, generator=g).to(torch.bfloat16).cuda()
    return q, kp, vp, table, torch.tensor(lens, dtype=torch.int32).cuda()


def exact(q, kp, vp, table, lens, window, sinks):
    q, kp, vp = (t.double().cpu().numpy() for t in (q, kp, vp))
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(lens):
        k, v = H.gather(kp, table[b].numpy(), n), H.gather(vp, table[b].numpy(), n)
        ok, scale = H.seen(1, n, window, sinks), q.shape[-1] ** -0.5
        out[b] = H.masked_fwd(q[b:b + 1], k, v, ok, scale)[0][0]
        spread[b] = H.masked_fwd(q[b:b + 1], k, np.abs(v), ok, scale)[0][0]
    return out, spread


# query heads up to 8 a K/V head, and more (another kernel); lengths whose softmax has a few large
# weights, and one that several CTAs share
@pytest.mark.parametrize("hq,hkv,dh", [(8, 8, 64), (8, 2, 128), (16, 2, 64), (12, 1, 128), (24, 1, 64), (32, 2, 128)])
@pytest.mark.parametrize("lens,window,sinks", [([2, 3, 5, 9, 17, 33, 63], 0, 0), ([40, 90, 700], 12, 2), ([20000], 0, 0)],
                         ids=["few", "window", "long"])
def test_decode_keeps_the_weights(hq, hkv, dh, lens, window, sinks):
    q, kp, vp, table, lt = make(7, lens, hq, hkv, dh)
    out, _ = ra.paged_attn_decode(q, ra.make_cache(kp, vp, table.cuda()), lt, window=window, sinks=sinks)
    assert ra.check_device_status() == 0, ra.last_error()
    ref, spread = exact(q, kp, vp, table, lens, window, sinks)
    err = np.abs(out.double().cpu().numpy() - ref)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -12 * spread
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size} off, worst {(err / tol).max():.2f} of the bound"


@pytest.mark.parametrize("hq", [4, 12])
def test_an_infinite_value_is_seen_as_one(hq):
    """A visible v of +-inf gives an infinite result in its column, and leaves the others alone."""
    q, kp, vp, table, lt = make(9, [50, 50], hq, 1, 64)
    cache = ra.make_cache(kp, vp, table.cuda())
    want, _ = ra.paged_attn_decode(q, cache, lt)
    vp[table[0, 1].item(), 3, 0, 5] = float("inf")
    vp[table[0, 2].item(), 1, 0, 60] = -float("inf")
    out, _ = ra.paged_attn_decode(q, cache, lt)
    assert (out[0, :, 5] == float("inf")).all() and (out[0, :, 60] == -float("inf")).all()
    out[0, :, [5, 60]] = want[0, :, [5, 60]]
    assert torch.equal(out, want)
