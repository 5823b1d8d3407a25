"""Refusals of the calls with positions on several axes (no GPU): invalid arguments are answered with the
right status before anything is launched. The pointers are never followed."""
import ctypes

import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from context_blockwise_attention_step_gb300 import _abi

FAKE = 256


@pytest.fixture(scope="module", autouse=True)
def built_library():
    ra.build()
    return _abi.lib()


def _prob(**kw):
    return ra.make_problem(**{**dict(dtype=torch.bfloat16, layout="zigzag", causal=True, D=4, hq=8, hkv=2, head_dim=128,
                                     batch=2, seqlen=64), **kw})


def test_sections():
    assert ra.axis_sections([2, 1, 3]) == [0, 0, 1, 2, 2, 2]
    assert ra.axis_sections([4, 2, 2], cyclic=True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert ra.axis_sections([3, 3], cyclic=True) == [0, 1, 0, 1, 0, 1]


def test_the_struct_holds_what_it_was_given():
    axis = [0, 1, 2, 0, 1, 2, 1, 1]
    one, many = ra.make_rope(16, base=50.0, interleaved=True), ra.make_axis_rope(16, axis, base=50.0, interleaved=True)
    assert list(many.raw.rope.turns) == list(one.raw.turns) and many.raw.rope.interleaved == 1
    assert many.raw.n_axes == 3 and list(many.raw.axis[:8]) == axis


def test_init_refusals():
    L, r = _abi.lib(), _abi.RaAxisRope()
    f, a = (ctypes.c_double * 2)(1.0, 0.25), (ctypes.c_int32 * 2)(0, 2)
    bad = _abi.RA_ERR_INVALID_ARG
    ok = lambda p=ctypes.byref(r), rd=4, f=f, n=3, a=a: L.ra_axis_rope_init(p, rd, 0, f, n, a)  # noqa: E731
    assert ok() == _abi.RA_OK
    for kw in (dict(p=None), dict(f=None), dict(a=None), dict(n=2), dict(n=0), dict(n=9), dict(rd=3), dict(rd=130),
               dict(a=(ctypes.c_int32 * 2)(0, -1)), dict(f=(ctypes.c_double * 2)(1.0, float("inf")))):
        assert ok(**kw) == bad, kw
    with pytest.raises(ValueError):
        ra.make_axis_rope(8, [0, 1, 2])
    with pytest.raises(ValueError):
        ra.make_axis_rope(8, [0, 1, 2, 8])
    with pytest.raises(ValueError):
        ra.make_axis_rope(8, [0, 1, 2, -1])


def test_call_refusals():
    L, p, rope = _abi.lib(), _prob(), ra.make_axis_rope(128, ra.axis_sections([16, 24, 24]))
    bad, shape = _abi.RA_ERR_INVALID_ARG, _abi.RA_ERR_SHAPE

    def fwd(rope=rope.ptr, pos=FAKE, stride=3, q=FAKE, qw=FAKE, p=p, eps=1e-6):
        return L.ra_qk_norm_axis_rope_fwd(p.ptr, rope, pos, stride, eps, q, 1024, FAKE, 256, qw, FAKE, 512, 512, None)

    def bwd(rope=rope.ptr, pos=FAKE, stride=3, q=FAKE, qw=FAKE, p=p, eps=1e-6):
        return L.ra_qk_norm_axis_rope_bwd(p.ptr, rope, pos, stride, eps, FAKE, FAKE, q, 1024, FAKE, 256, qw, FAKE, FAKE,
                                          FAKE, FAKE, FAKE, FAKE, 1 << 30, None)
    hand = _abi.RaAxisRope()  # filled in by hand: an axis that is not there
    ctypes.memmove(ctypes.byref(hand), ctypes.byref(rope.raw), ctypes.sizeof(hand))
    hand.axis[5] = 3
    for call in (fwd, bwd):
        assert call(rope=None) == bad
        assert call(pos=None) == bad
        assert call(stride=2) == shape
        assert call(stride=-3) == shape
        assert call(q=None) == bad
        assert call(qw=None) == bad
        assert call(eps=float("nan")) == bad
        assert call(rope=ctypes.byref(hand)) == bad
        assert call(rope=ctypes.byref(_abi.RaAxisRope())) == bad
        assert call(p=_prob(head_dim=64)) == shape
        assert call(p=_prob(D=0)) == bad

    c = _abi.RaPagedCache(_abi.RA_BF16, 2, 128, 16, 8, 3, 4, 4, 16 * 256, 256, 128, FAKE, FAKE, FAKE)

    def append(rope=rope.ptr, pos=FAKE, stride=3, k=FAKE, n=3):
        return L.ra_kv_cache_append_axes(ctypes.byref(c), rope, pos, stride, 1e-6, n, 8, FAKE, 1024, k, 256, FAKE, 256,
                                         None, None, FAKE, None, 512, None)
    assert append(rope=None) == bad
    assert append(pos=None) == bad
    assert append(stride=0) == shape
    assert append(k=None) == bad
    assert append(n=2) == shape
    assert append(rope=ctypes.byref(hand)) == bad


def test_positions_go_with_an_axis_rope():
    """(The tensors are on the CPU: what is refused is refused for its positions first, or for its device.)"""
    p = _prob()
    q, k = torch.zeros(2, 64, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 64, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ra.qk_norm_rope_fwd(q, k, p, rope=ra.make_rope(128), positions=torch.zeros(2, 64, 3, dtype=torch.int32))
    with pytest.raises(ValueError):
        ra.qk_norm_rope_fwd(q, k, p, rope=ra.make_axis_rope(128, ra.axis_sections([16, 24, 24])))
