"""bf16 token tensors that do not begin on 16 bytes are refused before anything is launched (no GPU;
the pointers are never followed). The tensor-core kernels copy and store 16 bytes at a time."""
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from context_blockwise_attention_step_gb300 import _abi

FAKE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built_library():
    ra.build()


def _prob(dtype=torch.bfloat16):
    return ra.make_problem(dtype=dtype, layout="zigzag", causal=True, D=4, hq=8, hkv=2, head_dim=128, batch=2, seqlen=64)


# per call: the positions of its token tensors among its pointers, and the pointers' number
@pytest.mark.parametrize("off", [2, 8])
@pytest.mark.parametrize("bad", [0, 1, 2, 3])
def test_forward_calls(bad, off):
    L, p = _abi.lib(), _prob()
    t = [FAKE] * 4
    t[bad] += off
    q, k, v, out = t
    for call in (lambda: L.ra_ring_attn_fwd(p.ptr, q, k, v, out, FAKE, None, 0, None),
                 lambda: L.ra_window_attn_fwd(p.ptr, 8, 2, q, k, v, out, FAKE, None, 0, None),
                 lambda: L.ra_window_attn_fwd(p.ptr, 64, 2, q, k, v, out, FAKE, None, 0, None),
                 lambda: L.ra_block_attn_fwd(p.ptr, -1, 0, q, k, v, out, _abi.RA_BF16, FAKE, None),
                 lambda: L.ra_block_attn_fwd(p.ptr, -1, 0, q, k, v, out, _abi.RA_F32, FAKE, None)):
        assert call() == _abi.RA_ERR_INVALID_ARG
        assert "aligned" in ra.last_error()


@pytest.mark.parametrize("bad", range(7))
def test_backward_calls(bad):
    L, p = _abi.lib(), _prob()
    t = [FAKE] * 7
    t[bad] += 8
    q, k, v, dout, dq, dk, dv = t
    for call in (lambda: L.ra_ring_attn_bwd(p.ptr, q, k, v, FAKE, FAKE, dout, dq, dk, dv, FAKE, 1 << 20, None),
                 lambda: L.ra_window_attn_bwd(p.ptr, 8, 2, q, k, v, FAKE, FAKE, dout, dq, dk, dv, FAKE, 1 << 30, None),
                 lambda: L.ra_block_attn_bwd(p.ptr, -1, 0, q, k, v, FAKE, FAKE, dout, dq, dk, dv, FAKE, 1 << 20, None)):
        assert call() == _abi.RA_ERR_INVALID_ARG
        assert "aligned" in ra.last_error()
