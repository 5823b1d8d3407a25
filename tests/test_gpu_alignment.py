"""Tensors that begin on any element: refused where the kernels move 16 bytes at a time, and elsewhere
the same results as on aligned ones."""
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from context_blockwise_attention_step_gb300 import _abi

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


def shifted(t):
    """A copy of t that begins one element behind an allocation's start."""
    x = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
    return x.copy_(t)


def make(dt):
    g = torch.Generator().manual_seed(3)
    x = [torch.randn(2, 96, h, 64, generator=g).to(dt).cuda() for h in (4, 2, 2, 4)]
    return x, ra.problem_for(x[0], x[1], D=2, layout="zigzag")


def test_bf16_attention_refuses_them():
    (q, k, v, do), prob = make(BF16)
    out, lse = ra.window_attn_fwd(q, k, v, prob, 20, 1)
    for window in (20, 96):  # (the second is the ring call)
        for call in (lambda: ra.window_attn_fwd(q, k, v, prob, window, 1, out=shifted(out)),
                     lambda: ra.window_attn_fwd(shifted(q), k, v, prob, window, 1),
                     lambda: ra.window_attn_bwd(do, q, k, v, out, lse, prob, window, 1, dk=shifted(k)),
                     lambda: ra.window_attn_bwd(shifted(do), q, k, v, out, lse, prob, window, 1)):
            with pytest.raises(ra.RingAttnError) as e:
                call()
            assert e.value.status == _abi.RA_ERR_INVALID_ARG
    with pytest.raises(ra.RingAttnError):
        ra.ring_attn_fwd(q, k, v, prob, out=shifted(out))
    grads = ra.window_attn_bwd(do, q, k, v, out, lse, prob, 20, 1)
    again = ra.window_attn_bwd(do, q, k, v, shifted(out), lse, prob, 20, 1)  # the forward's out alone may
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_float32_attention_takes_them():
    (q, k, v, do), prob = make(F32)
    out, lse = ra.window_attn_fwd(q, k, v, prob, 20, 1)
    grads = ra.window_attn_bwd(do, q, k, v, out, lse, prob, 20, 1)
    q2, k2, v2, do2, out2 = (shifted(t) for t in (q, k, v, do, torch.zeros_like(out)))
    o, l = ra.window_attn_fwd(q2, k2, v2, prob, 20, 1, out=out2)
    assert torch.equal(o, out) and torch.equal(l, lse)
    g = ra.window_attn_bwd(do2, q2, k2, v2, o, l, prob, 20, 1, dq=shifted(q), dk=shifted(k), dv=shifted(v))
    assert all(torch.equal(a, b) for a, b in zip(g, grads))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_merge_takes_them(dt):
    (q, k, v, _), prob = make(BF16)
    block, blse = ra.block_attn_fwd(q, k, v, prob, -1, 1, out_dtype=dt)
    res = []
    for make_out, b in ((lambda t: t, block), (shifted, block), (lambda t: t, shifted(block)), (shifted, shifted(block))):
        out, lse = ra.block_attn_fwd(q, k, v, prob, -1, 0)
        out = make_out(out)
        res.append(ra.update_out_and_lse(out, lse, b, blse, prob))
    for out, lse in res[1:]:
        assert torch.equal(out, res[0][0]) and torch.equal(lse, res[0][1])
