"""Refusals of the head-norm, paged-cache and decode calls (no GPU): invalid arguments are
answered with the right status before anything is launched. The pointers are never followed."""
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
    base = dict(dtype=torch.bfloat16, layout="zigzag", causal=True, D=4, hq=8, hkv=2, head_dim=128,
                batch=2, seqlen=64)
    base.update(kw)
    return ra.make_problem(**base)


def _cache(**kw):
    c = _abi.RaPagedCache()
    base = dict(dtype=_abi.RA_BF16, hkv=2, head_dim=128, page_size=16, n_pages=8, n_seqs=3, max_pages=4,
                table_stride=4, page_stride=16 * 256, slot_stride=256, head_stride=128, k_pages=FAKE,
                v_pages=FAKE, block_table=FAKE)
    base.update(kw)
    for k, v in base.items():
        setattr(c, k, v)
    return c


def test_rope_init_refusals_and_turns():
    L = _abi.lib()
    r = _abi.RaRope()
    f = (ctypes.c_double * 2)(1.0, 0.25)
    for rd in (0, 1, 3, 130, -2):
        assert L.ra_rope_init(ctypes.byref(r), rd, 0, f) == _abi.RA_ERR_INVALID_ARG
    assert L.ra_rope_init(None, 4, 0, f) == _abi.RA_ERR_INVALID_ARG
    assert L.ra_rope_init(ctypes.byref(r), 4, 0, None) == _abi.RA_ERR_INVALID_ARG
    bad = (ctypes.c_double * 2)(1.0, float("nan"))
    assert L.ra_rope_init(ctypes.byref(r), 4, 0, bad) == _abi.RA_ERR_INVALID_ARG
    two_pi = 6.283185307179586
    f = (ctypes.c_double * 3)(two_pi / 4, -two_pi / 4, 3 * two_pi)
    assert L.ra_rope_init(ctypes.byref(r), 6, 1, f) == _abi.RA_OK
    assert r.rotary_dim == 6 and r.interleaved == 1
    # a quarter turn, three quarters, whole turns (none), within double rounding
    for got, want in zip(r.turns[:3], (1 << 62, 3 << 62, 0)):
        assert min((got - want) % 2 ** 64, (want - got) % 2 ** 64) < 2 ** 14
    with pytest.raises(ValueError):
        ra.make_rope(7)
    with pytest.raises(ValueError):
        ra.make_rope(8, inv_freq=[1.0, 2.0])


def _fwd(p, rope=None, eps=1e-6, q=FAKE, qs=8 * 128, k=FAKE, ks=2 * 128, qw=FAKE, kw=FAKE, qo=512, ko=512):
    return _abi.lib().ra_qk_norm_rope_fwd(p.ptr, rope, eps, q, qs, k, ks, qw, kw, qo, ko, None)


def test_norm_rope_refusals():
    p = _prob()
    rope = ra.make_rope(128)
    for null in ("q", "k", "qo", "ko"):
        assert _fwd(p, **{null: None}) == _abi.RA_ERR_INVALID_ARG
    assert _fwd(p, kw=None) == _abi.RA_ERR_INVALID_ARG
    assert _fwd(p, qw=None, kw=None) == _abi.RA_ERR_INVALID_ARG  # nothing to do
    assert _fwd(p, eps=float("nan")) == _abi.RA_ERR_INVALID_ARG
    assert _fwd(p, eps=-1.0) == _abi.RA_ERR_INVALID_ARG
    assert _fwd(p, qs=8 * 128 - 1) == _abi.RA_ERR_SHAPE
    assert _fwd(p, ks=0) == _abi.RA_ERR_SHAPE
    assert _fwd(p, qo=FAKE, qs=8 * 128 + 8) == _abi.RA_ERR_INVALID_ARG  # strided, in place
    small = _prob(head_dim=64)
    assert _fwd(small, rope=rope.ptr) == _abi.RA_ERR_SHAPE
    assert _fwd(_prob(D=0)) == _abi.RA_ERR_INVALID_ARG
    empty = _abi.RaRope()
    assert _fwd(p, rope=ctypes.byref(empty)) == _abi.RA_ERR_INVALID_ARG
    L = _abi.lib()
    need = ra.workspace_bytes(p, 3)
    assert need >= 2 * 128 * 4

    def bwd(ws=FAKE, size=need, dqw=FAKE, q=FAKE):
        return L.ra_qk_norm_rope_bwd(p.ptr, rope.ptr, 1e-6, FAKE, FAKE, q, 1024, FAKE, 256, FAKE, FAKE, FAKE,
                                     FAKE, dqw, FAKE, ws, size, None)
    assert bwd(size=need - 1) == _abi.RA_ERR_WORKSPACE
    assert bwd(ws=None) == _abi.RA_ERR_INVALID_ARG
    assert bwd(ws=128) == _abi.RA_ERR_INVALID_ARG
    assert bwd(dqw=None) == _abi.RA_ERR_INVALID_ARG
    assert bwd(q=None) == _abi.RA_ERR_INVALID_ARG


BAD_CACHES = [
    (dict(dtype=7), _abi.RA_ERR_INVALID_ARG), (dict(hkv=0), _abi.RA_ERR_INVALID_ARG),
    (dict(page_size=0), _abi.RA_ERR_INVALID_ARG), (dict(n_pages=0), _abi.RA_ERR_INVALID_ARG),
    (dict(n_seqs=-1), _abi.RA_ERR_INVALID_ARG), (dict(max_pages=-1), _abi.RA_ERR_INVALID_ARG),
    (dict(head_dim=96), _abi.RA_ERR_UNSUPPORTED),
    (dict(dtype=_abi.RA_F32, head_dim=129), _abi.RA_ERR_UNSUPPORTED),
    (dict(n_seqs=_abi.RA_MAX_CACHE_SEQS + 1), _abi.RA_ERR_UNSUPPORTED),
    (dict(max_pages=1 << 28, table_stride=1 << 28), _abi.RA_ERR_UNSUPPORTED),
    (dict(table_stride=3), _abi.RA_ERR_INVALID_ARG), (dict(slot_stride=0), _abi.RA_ERR_INVALID_ARG),
    (dict(page_stride=-16), _abi.RA_ERR_INVALID_ARG), (dict(k_pages=None), _abi.RA_ERR_INVALID_ARG),
    (dict(block_table=None), _abi.RA_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES, ids=lambda x: str(x))
def test_bad_caches_are_refused_by_append_and_decode(kw, status):
    L, c = _abi.lib(), _cache(**kw)
    p = ctypes.byref(c)
    assert L.ra_kv_cache_append(p, None, 0.0, 3, 8, FAKE, 1024, FAKE, 256, FAKE, 256, None, None, FAKE, None,
                                FAKE, None) == status
    assert L.ra_paged_attn_decode(p, 8, 0.0, 0, 0, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == status
    assert L.ra_paged_workspace_bytes(p, 8) == 0


def test_append_and_decode_refusals():
    L, c = _abi.lib(), _cache()
    p = ctypes.byref(c)

    def append(n=3, hq=8, q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, qw=None, kw=None, lens=FAKE, qo=512,
               rope=None):
        return L.ra_kv_cache_append(p, rope, 1e-6, n, hq, q, qs, k, ks, v, vs, qw, kw, lens, None, qo, None)
    assert append(n=2) == _abi.RA_ERR_SHAPE
    assert append(n=-1) == _abi.RA_ERR_INVALID_ARG
    assert append(hq=7) == _abi.RA_ERR_UNSUPPORTED
    assert append(q=None) == _abi.RA_ERR_INVALID_ARG
    assert append(qo=None) == _abi.RA_ERR_INVALID_ARG
    for name in ("k", "v", "lens"):
        assert append(**{name: None}) == _abi.RA_ERR_INVALID_ARG
    for name in ("qs", "ks", "vs"):
        assert append(**{name: 8}) == _abi.RA_ERR_SHAPE
    assert append(qw=FAKE) == _abi.RA_ERR_INVALID_ARG
    assert append(qo=FAKE, qs=2048) == _abi.RA_ERR_INVALID_ARG

    need = L.ra_paged_workspace_bytes(p, 8)
    assert need > 0

    def decode(hq=8, scale=0.0, window=0, sinks=0, q=FAKE, lens=FAKE, out=FAKE, lse=FAKE, ws=FAKE, size=need):
        return L.ra_paged_attn_decode(p, hq, scale, window, sinks, q, lens, out, lse, ws, size, None)
    assert decode(hq=3) == _abi.RA_ERR_UNSUPPORTED
    assert decode(hq=0) == _abi.RA_ERR_UNSUPPORTED
    assert decode(scale=float("inf")) == _abi.RA_ERR_INVALID_ARG
    assert decode(window=-1) == _abi.RA_ERR_INVALID_ARG
    assert decode(window=4, sinks=-1) == _abi.RA_ERR_INVALID_ARG
    for name in ("q", "lens", "out", "lse", "ws"):
        assert decode(**{name: None}) == _abi.RA_ERR_INVALID_ARG
    assert decode(size=need - 1) == _abi.RA_ERR_WORKSPACE
    assert decode(ws=64) == _abi.RA_ERR_INVALID_ARG
    assert ra.last_error() != ""


def test_python_checks_need_cuda_tensors():
    k = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ra.make_cache(k, k, torch.zeros(3, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        ra.make_cache(k, k.float(), torch.zeros(3, 4, dtype=torch.int32))
    q = torch.zeros(2, 64, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ra.qk_norm_rope_fwd(q, q[:, :, :2], _prob(), rope=ra.make_rope(128))


def test_window_refusals():
    L, p = _abi.lib(), _prob()

    def fwd(p=p, window=8, sinks=0, q=FAKE, ws=None, size=0):
        return L.ra_window_attn_fwd(p.ptr, window, sinks, q, FAKE, FAKE, FAKE, FAKE, ws, size, None)
    assert fwd(window=0) == _abi.RA_ERR_INVALID_ARG
    assert fwd(window=-5) == _abi.RA_ERR_INVALID_ARG
    assert fwd(sinks=-1) == _abi.RA_ERR_INVALID_ARG
    assert fwd(sinks=_abi.RA_MAX_SINKS + 1) == _abi.RA_ERR_INVALID_ARG
    assert fwd(p=_prob(causal=False)) == _abi.RA_ERR_UNSUPPORTED
    assert fwd(p=_prob(seqlen=60)) == _abi.RA_ERR_SHAPE
    assert fwd(p=_prob(D=65, layout="basic", seqlen=650)) == _abi.RA_ERR_UNSUPPORTED
    assert fwd(q=None) == _abi.RA_ERR_INVALID_ARG
    assert fwd(ws=64, size=1024) == _abi.RA_ERR_INVALID_ARG
    assert fwd(window=1 << 30, q=None) == _abi.RA_ERR_INVALID_ARG  # the ring call's refusals
    need = ra.window_workspace_bytes(p, 8, 4, 1)
    assert need >= ra.workspace_bytes(p, 2)
    assert ra.window_workspace_bytes(p, 0, 0, 1) == 0

    def bwd(window=8, sinks=4, ws=FAKE, size=need, dq=FAKE):
        return L.ra_window_attn_bwd(p.ptr, window, sinks, *([FAKE] * 6), dq, FAKE, FAKE, ws, size, None)
    assert bwd(size=need - 1) == _abi.RA_ERR_WORKSPACE
    assert bwd(ws=None) == _abi.RA_ERR_INVALID_ARG
    assert bwd(ws=128) == _abi.RA_ERR_INVALID_ARG
    assert bwd(dq=None) == _abi.RA_ERR_INVALID_ARG
    assert bwd(window=0) == _abi.RA_ERR_INVALID_ARG


def test_window_workspace(monkeypatch):
    """The slots of the sinks' sums stay small beside the tensors: a slot holds the sink rows of one
    shard, and a sequence has about as many slots as windows, or 64."""
    rows, hkv, dh = 131072, 8, 128
    for dt, layout, D in ((torch.bfloat16, "zigzag", 16), (torch.bfloat16, "stripe", 64), (torch.float32, "stripe", 64),
                          (torch.float32, "basic", 1)):
        p = _prob(dtype=dt, layout=layout, D=D, hq=32, hkv=hkv, batch=1, seqlen=rows)
        plain = ra.window_workspace_bytes(p, 1024, 0)
        kv = 2 * rows * hkv * dh * (2 if dt == torch.bfloat16 else 4)
        assert 0 < ra.window_workspace_bytes(p, 1024, 128) - plain < kv
        assert ra.window_workspace_bytes(p, 1024, 4) - plain < kv // 8
        assert ra.window_workspace_bytes(p, 1024, 4, 0) == ra.workspace_bytes(p, 0)
    p = _prob()
    monkeypatch.setenv("RA_BWD", "fused")  # a window over everything is the ring call, with its workspace
    assert ra.window_workspace_bytes(p, 64, 4, 1) == ra.workspace_bytes(p, 1)


def test_window_of_no_tokens():
    L, p = _abi.lib(), _prob(batch=0, cu_seqlens=[0, 0, 0])
    assert L.ra_window_attn_fwd(p.ptr, 8, 2, *([None] * 6), 0, None) == _abi.RA_OK
    assert L.ra_window_attn_bwd(p.ptr, 8, 2, *([None] * 10), 0, None) == _abi.RA_OK
