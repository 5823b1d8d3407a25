"""Problems of no tokens: a batch whose every sequence is idle."""
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from context_blockwise_attention_step_gb300 import _abi


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()


@pytest.mark.parametrize("cu", [[0], [0, 0, 0]])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_ring_calls_of_no_tokens(cu, dt):
    L = _abi.lib()
    p = ra.make_problem(dtype=dt, layout="zigzag", causal=True, D=2, hq=4, hkv=2, head_dim=64, cu_seqlens=cu)
    assert L.ra_ring_attn_fwd(p.ptr, *([None] * 6), 0, None) == _abi.RA_OK
    assert L.ra_ring_attn_bwd(p.ptr, *([None] * 10), 0, None) == _abi.RA_OK
    assert L.ra_window_attn_fwd(p.ptr, 8, 2, *([None] * 6), 0, None) == _abi.RA_OK
    assert L.ra_window_attn_bwd(p.ptr, 8, 2, *([None] * 10), 0, None) == _abi.RA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(window=9, sinks=1), dict(qk_norm=True, rope=None)], ids=str)
def test_prefill_and_decode_of_idle_sequences(kw):
    m = ra.RingSelfAttention(96, 4, 2, 64, D=2, device="cuda", **{"rope": ra.make_rope(64), **kw})
    pages = torch.full((2, 3, 16, 2, 64), 7.0, device="cuda").bfloat16()
    cache = ra.make_cache(pages[0], pages[1], torch.zeros(2, 1, dtype=torch.int32, device="cuda"))
    y = m.prefill(torch.empty(0, 96, device="cuda").bfloat16(), cache, [0, 0, 0])
    assert y.shape == (0, 96)
    y = m.decode(torch.randn(2, 96, device="cuda").bfloat16(), cache, torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert (y == 0).all() and (pages == 7).all()
    assert ra.check_device_status() == 0
