"""What moves tokens between orders reads device memory only: tensors on the host are refused before
anything is launched (no GPU)."""
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra


@pytest.fixture(scope="module", autouse=True)
def built_library():
    ra.build()


def test_host_tensors_are_refused():
    prob = ra.make_problem(dtype=torch.bfloat16, layout="zigzag", causal=True, D=2, hq=2, hkv=1, head_dim=64, batch=1,
                           seqlen=8)
    x = torch.zeros(1, 8, 3, dtype=torch.int32)
    for move in (ra.shard_tokens, ra.unshard_tokens):
        with pytest.raises(ValueError):
            move(x, prob)
        with pytest.raises(ValueError):
            move(x, prob, out=torch.empty_like(x))


def test_the_layer_wants_positions_where_x_is():
    m = ra.RingSelfAttention(32, 2, 1, 64, D=2, device="meta", rope=ra.make_axis_rope(64, [0, 1] * 16))
    x = torch.zeros(1, 8, 32, device="meta", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="positions must be on meta"):
        m(x, torch.zeros(1, 8, 2, dtype=torch.int32))
