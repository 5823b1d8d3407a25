"""Second derivatives: refused where there is no formula for them, right where there is."""
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


def inputs(dt):
    g = torch.Generator().manual_seed(11)
    q, k, v = (torch.randn(1, 64, h, 64, generator=g).to(dt).cuda().requires_grad_() for h in (4, 2, 2))
    return q, k, v, ra.problem_for(q, k, D=2, layout="zigzag")


@pytest.mark.parametrize("dt", [BF16, F32])
def test_attention_and_norm_refuse_a_second_derivative(dt):
    q, k, v, prob = inputs(dt)
    w = torch.ones(64, dtype=dt, device="cuda", requires_grad=True)
    calls = (lambda: ra.ring_attention(q, k, v, prob)[0], lambda: ra.ring_attention(q, k, v, prob, window=9, sinks=1)[0],
             lambda: ra.qk_norm_rope(q, k, prob, w, w, ra.make_rope(64))[0],
             lambda: ra.qk_norm_rope(q, k, prob, rope=ra.make_rope(64))[0])
    for call in calls:
        first = torch.autograd.grad(call().float().square().sum(), q)[0]
        again = torch.autograd.grad(call().float().square().sum(), q, create_graph=True)[0]
        assert torch.equal(first, again)  # the gradient itself is there with a graph too
        with pytest.raises(RuntimeError, match="once_differentiable"):
            again.float().square().sum().backward()


@pytest.mark.parametrize("move,back", [(ra.shard, ra.unshard), (ra.unshard, ra.shard)])
def test_permutations_have_every_derivative(move, back):
    x, _, _, prob = inputs(F32)
    g = torch.autograd.grad(move(x, prob).pow(3).sum(), x, create_graph=True)[0]
    assert torch.equal(g, 3 * x.detach() ** 2)
    h = torch.autograd.grad((g * x.detach()).sum(), x)[0]
    assert (h - 6 * x.detach() ** 2).abs().max() <= 1e-5 * x.detach().abs().max() ** 2
