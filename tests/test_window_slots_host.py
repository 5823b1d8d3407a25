"""The sinks' sums of a windowed backward over very many shards and heads (no GPU; the pointers are
never followed): a size that 32 bits do not count is refused, not wrapped to a small workspace."""
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from context_blockwise_attention_step_gb300 import _abi

FAKE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built_library():
    ra.build()


@pytest.mark.parametrize("D,h", [(32768, 512), (32768, 1024), (65536, 1024), (1 << 20, 64)])
@pytest.mark.parametrize("layout", ["basic", "stripe"])
def test_more_slots_than_32_bits_count(D, h, layout):
    """D shards of one token, `h` heads, 128 sinks: 128 h (1 + D) slots."""
    L = _abi.lib()
    p = ra.make_problem(dtype=torch.float32, layout=layout, causal=True, D=D, hq=h, hkv=h, head_dim=1, batch=1, seqlen=D)
    assert ra.validate(p) == _abi.RA_OK and 128 * h * (1 + D) >= 2 ** 31
    assert ra.window_workspace_bytes(p, 1, 128, 1) == 0
    st = L.ra_window_attn_bwd(p.ptr, 1, 128, *([FAKE] * 9), FAKE, 1 << 62, None)
    assert st == _abi.RA_ERR_UNSUPPORTED
    few = ra.window_workspace_bytes(p, 1, 1, 1)  # one sink: h (1 + D) slots of two floats
    assert few >= h * (1 + D) * 2 * 4 + D * h * 4
    st = L.ra_window_attn_bwd(p.ptr, 1, 1, *([FAKE] * 9), FAKE, few - 1, None)
    assert st == _abi.RA_ERR_WORKSPACE


def test_the_largest_count_that_fits():
    D, h = 32767, 500  # 128 * 500 * 32768 slots, and 16 million items more, are below 2^31
    p = ra.make_problem(dtype=torch.float32, layout="basic", causal=True, D=D, hq=h, hkv=h, head_dim=1, batch=1, seqlen=D)
    assert ra.window_workspace_bytes(p, 1, 128, 1) >= 128 * h * (1 + D) * 2 * 4
