"""First tokens spread over many shards, with many K/V heads: more of both together than a launch's
second dimension has."""
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


def test_many_heads_are_the_heads_one_half_at_a_time():
    D, n, h, dh, window, sinks = 128, 256, 512, 4, 3, 128
    g = torch.Generator().manual_seed(2)
    x = [torch.randn(1, n, h, dh, generator=g).cuda() for _ in range(4)]

    def run(heads):
        t = [y[:, :, heads].contiguous() for y in x]
        prob = ra.problem_for(t[0], t[1], D=D, layout="stripe")
        q, k, v, do = (ra.shard_tokens(y, prob) for y in t)
        out, lse = ra.window_attn_fwd(q, k, v, prob, window, sinks)
        return out, *ra.window_attn_bwd(do, q, k, v, out, lse, prob, window, sinks)
    whole = run(slice(None))
    for heads in (slice(0, 256), slice(256, 512)):
        for a, b in zip(run(heads), whole):
            assert torch.equal(a, b[:, :, heads])
