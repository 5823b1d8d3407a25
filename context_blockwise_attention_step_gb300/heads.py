"""Head norms, the rotation by position, the sliding window, and the serving path: a paged
key-value cache and the attention of one or several new tokens over it, with prefixes that sequences
share (include/ringattn.h has the definitions).

Like ``ops``, this is a binding: every step runs in the library's kernels on the current (or a
given) stream, outputs are allocated unless they are passed in.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import ops
from ._abi import (RA_BF16, RA_F32, RA_MAX_AXES, RA_MAX_ROTARY_DIM, RaAxisRope, RaPagedCache, RaRope,
                   RaSharedPrefix, check, lib)
from .ops import Problem


@dataclass
class Rope:
    """A rotation by position; ``raw`` is the C struct handed to the library."""

    raw: RaRope

    def __post_init__(self):
        self.ptr = ctypes.byref(self.raw)


def make_rope(rotary_dim: int, base: float = 10000.0, inv_freq=None, interleaved: bool = False) -> Rope:
    """The rotation of the first ``rotary_dim`` elements of a head: pair i turns by position *
    ``inv_freq[i]`` radians (default base ** (-2i / rotary_dim)). Pairs are (i, i +
    rotary_dim/2), or (2i, 2i+1) if ``interleaved``."""
    inv_freq = _inv_freq(rotary_dim, base, inv_freq)
    raw = RaRope()
    check(lib().ra_rope_init(ctypes.byref(raw), rotary_dim, 1 if interleaved else 0, inv_freq))
    return Rope(raw)


def _inv_freq(rotary_dim: int, base: float, inv_freq):
    if rotary_dim % 2 or not 2 <= rotary_dim <= RA_MAX_ROTARY_DIM:
        raise ValueError(f"rotary_dim must be even, 2..{RA_MAX_ROTARY_DIM}, got {rotary_dim}")
    if inv_freq is None:
        inv_freq = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if isinstance(inv_freq, torch.Tensor):
        inv_freq = inv_freq.detach().cpu().tolist()
    inv_freq = [float(x) for x in inv_freq]
    if len(inv_freq) != rotary_dim // 2:
        raise ValueError(f"inv_freq has {len(inv_freq)} entries, expected {rotary_dim // 2}")
    return (ctypes.c_double * len(inv_freq))(*inv_freq)


@dataclass
class AxisRope:
    """A rotation of tokens with positions on several axes; ``raw`` is the C struct handed to the
    library. The calls that take it take the tokens' ``positions`` too."""

    raw: RaAxisRope

    def __post_init__(self):
        self.ptr = ctypes.byref(self.raw)
        self.n_axes = self.raw.n_axes


def make_axis_rope(rotary_dim: int, axis, base: float = 10000.0, inv_freq=None,
                   interleaved: bool = False) -> AxisRope:
    """``make_rope`` for tokens that have a position on each of several axes: pair i turns by the
    position on axis ``axis[i]`` (rotary_dim/2 integers, see ``axis_sections``) * ``inv_freq[i]``
    radians."""
    inv_freq = _inv_freq(rotary_dim, base, inv_freq)
    if isinstance(axis, torch.Tensor):
        axis = axis.detach().cpu().tolist()
    axis = [int(a) for a in axis]
    if len(axis) != rotary_dim // 2:
        raise ValueError(f"axis has {len(axis)} entries, expected {rotary_dim // 2}")
    n_axes = max(axis) + 1
    if min(axis) < 0 or n_axes > RA_MAX_AXES:
        raise ValueError(f"axis must hold numbers from 0 to {RA_MAX_AXES - 1}, got {min(axis)}..{max(axis)}")
    raw = RaAxisRope()
    check(lib().ra_axis_rope_init(ctypes.byref(raw), rotary_dim, 1 if interleaved else 0, inv_freq, n_axes,
                                  (ctypes.c_int32 * len(axis))(*axis)))
    return AxisRope(raw)


def axis_sections(sections, cyclic: bool = False) -> list:
    """The axis of every pair for ``make_axis_rope``: the first sections[0] pairs on axis 0, the next
    sections[1] on axis 1, and so on; or, ``cyclic``, the axes in turn (pair i on axis i % n as long
    as that axis has pairs left by its section: i < n * sections[i % n], else on axis 0). The turns end
    with the pairs: where a + n * (sections[a] - 1) is not below their number, axis a > 0 gets fewer than
    its section ([10, 20, 20] gives 17, 17 and 16)."""
    sections = [int(x) for x in sections]
    n = len(sections)
    if not cyclic:
        return [a for a, s in enumerate(sections) for _ in range(s)]
    return [i % n if i < n * sections[i % n] else 0 for i in range(sum(sections))]


def _rows(t: torch.Tensor, name: str, dtype, rows: int, heads: int, dh: int, dev: int) -> int:
    """Checks a token tensor [rows, heads, dh] or [B, S, heads, dh], possibly a view into a
    wider one, and returns the elements from one token to the next."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be on the same CUDA device as the other tensors")
    size = t.shape
    n = len(size)
    if n not in (3, 4) or size[-1] != dh or size[-2] != heads or t.numel() != rows * heads * dh:
        raise ValueError(f"{name} has shape {tuple(size)}, expected {rows} tokens of {heads} x {dh}")
    if t.is_contiguous():
        return heads * dh
    stride = t.stride()
    if (dh > 1 and stride[-1] != 1) or (heads > 1 and stride[-2] != dh):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    tokens = [(size[i], stride[i]) for i in range(n - 2) if size[i] > 1]
    if len(tokens) == 2 and tokens[0][1] != tokens[1][0] * tokens[1][1]:
        raise ValueError(f"{name}: batch elements must follow one another")
    return tokens[-1][1] if tokens and rows > 0 else heads * dh


def _plain(t: torch.Tensor, name: str, dtype, shape, dev: int) -> torch.Tensor:
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on CUDA device "
                         f"{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t


def _token(t: torch.Tensor, numel: int, name: str, prob: Problem, dev: int):
    if t.dtype != prob.token_dtype or t.numel() != numel or t.get_device() != dev or dev < 0 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {prob.token_dtype} tensor of {numel} elements on CUDA "
                         f"device {dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _weights(q_weight, k_weight, dtype, dh, dev):
    if (q_weight is None) != (k_weight is None):
        raise ValueError("pass both q_weight and k_weight, or neither")
    if q_weight is not None:
        _plain(q_weight, "q_weight", dtype, (dh,), dev)
        _plain(k_weight, "k_weight", dtype, (dh,), dev)


def _made_like(t: torch.Tensor, made: list) -> torch.Tensor:
    made.append(new := torch.empty_like(t, memory_format=torch.contiguous_format))
    return new


def _workspace(workspace, need: int, like: torch.Tensor, made: list):
    """The given workspace, or a new one on ``like``'s device (None if none is needed); and its bytes."""
    if workspace is None:
        if need > 0:
            made.append(workspace := torch.empty(need, device=like.device, dtype=torch.uint8))
        return workspace, need
    if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {like.device}")
    return workspace, workspace.numel() * workspace.element_size()


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _launch(dev: int, stream, made, call):
    """Runs ``call(stream handle)`` with device ``dev`` current. Tensors made for the call come
    from the current stream's pool: another ``stream`` waits for that stream first, and keeps
    them from reuse until it has done with them."""
    if stream is None and dev == torch.cuda.current_device():
        return check(call(torch._C._cuda_getCurrentRawStream(dev)))
    with torch.cuda.device(dev):
        if stream is None:
            return check(call(torch.cuda.current_stream().cuda_stream))
        if made and stream != torch.cuda.current_stream():
            stream.wait_stream(torch.cuda.current_stream())
            for t in made:
                t.record_stream(stream)
        return check(call(stream.cuda_stream))


def _rope_ptr(rope: Rope | None):
    return None if rope is None else rope.ptr


def _positions(rope, positions, rows: int, dev: int):
    """Whether the rotation takes positions on several axes, and the elements from one row's to the next."""
    if not isinstance(rope, AxisRope):
        if positions is not None:
            raise ValueError("positions go with a rotation on several axes (make_axis_rope)")
        return False, 0
    if positions is None:
        raise ValueError("a rotation on several axes wants positions")
    n = rope.n_axes
    if positions.dim() not in (2, 3):
        raise ValueError(f"positions must be [rows, {n}] or [B, S, {n}]")
    if (positions.dtype == torch.int32 and positions.is_contiguous() and positions.get_device() == dev
            and positions.shape[-1] == n and positions.numel() == rows * n):
        return True, n
    return True, _rows(positions.unsqueeze(-2), "positions", torch.int32, rows, 1, n, dev)


def qk_norm_rope_fwd(q, k, prob: Problem, q_weight=None, k_weight=None, rope: Rope | AxisRope | None = None,
                     eps: float = 1e-6, q_out=None, k_out=None, stream=None, positions=None):
    """Per-head root-mean-square norm (weights [head_dim] in the token dtype, or None for no
    norm) and rotation by global position (or None for no rotation) of shard-major q and k ->
    (q_out, k_out). q and k may be views into a wider tensor (a fused projection); q_out may be
    a contiguous q, k_out a contiguous k. With an ``AxisRope`` the rotation goes by ``positions``
    (int32, [rows, n_axes] or [B, S, n_axes], shard-major like q and k)."""
    r = prob.raw
    dh, dev = r.head_dim, q.get_device()
    qs = _rows(q, "q", prob.token_dtype, prob.rows, r.hq, dh, dev)
    ks = _rows(k, "k", prob.token_dtype, prob.rows, r.hkv, dh, dev)
    _weights(q_weight, k_weight, prob.token_dtype, dh, dev)
    made = []
    q_out = _made_like(q, made) if q_out is None else _plain(q_out, "q_out", prob.token_dtype, q.shape, dev)
    k_out = _made_like(k, made) if k_out is None else _plain(k_out, "k_out", prob.token_dtype, k.shape, dev)
    axes, ps = _positions(rope, positions, prob.rows, dev)
    rest = (eps, _ptr(q), qs, _ptr(k), ks, _ptr(q_weight), _ptr(k_weight), _ptr(q_out), _ptr(k_out))
    if axes:
        _launch(dev, stream, made, lambda s: lib().ra_qk_norm_axis_rope_fwd(prob.ptr, rope.ptr, _ptr(positions), ps,
                                                                            *rest, s))
    else:
        _launch(dev, stream, made, lambda s: lib().ra_qk_norm_rope_fwd(prob.ptr, _rope_ptr(rope), *rest, s))
    return q_out, k_out


def qk_norm_rope_bwd(dq_out, dk_out, q, k, prob: Problem, q_weight=None, k_weight=None,
                     rope: Rope | AxisRope | None = None, eps: float = 1e-6, dq=None, dk=None, workspace=None,
                     stream=None, positions=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of ``qk_norm_rope_fwd`` at its inputs q and k
    from those of its outputs. The weight gradients are float32 (None without weights), summed
    in a fixed order. dq may be dq_out, dk may be dk_out. ``positions`` as there."""
    r = prob.raw
    dh, dev = r.head_dim, dq_out.get_device()
    _plain(dq_out, "dq_out", prob.token_dtype, q.shape, dev)
    _plain(dk_out, "dk_out", prob.token_dtype, k.shape, dev)
    qs = _rows(q, "q", prob.token_dtype, prob.rows, r.hq, dh, dev)
    ks = _rows(k, "k", prob.token_dtype, prob.rows, r.hkv, dh, dev)
    _weights(q_weight, k_weight, prob.token_dtype, dh, dev)
    made = []
    dq = _made_like(q, made) if dq is None else _plain(dq, "dq", prob.token_dtype, q.shape, dev)
    dk = _made_like(k, made) if dk is None else _plain(dk, "dk", prob.token_dtype, k.shape, dev)
    dqw = dkw = None
    size = 0
    if q_weight is not None:
        made.append(dqw := torch.empty(dh, device=dq_out.device, dtype=torch.float32))
        made.append(dkw := torch.empty(dh, device=dq_out.device, dtype=torch.float32))
        workspace, size = _workspace(workspace, workspace is None and ops.workspace_bytes(prob, 3), q, made)
    axes, ps = _positions(rope, positions, prob.rows, dev)
    rest = (eps, _ptr(dq_out), _ptr(dk_out), _ptr(q), qs, _ptr(k), ks, _ptr(q_weight), _ptr(k_weight), _ptr(dq),
            _ptr(dk), _ptr(dqw), _ptr(dkw), _ptr(workspace), size)
    if axes:
        _launch(dev, stream, made, lambda s: lib().ra_qk_norm_axis_rope_bwd(prob.ptr, rope.ptr, _ptr(positions), ps,
                                                                            *rest, s))
    else:
        _launch(dev, stream, made, lambda s: lib().ra_qk_norm_rope_bwd(prob.ptr, _rope_ptr(rope), *rest, s))
    return dq, dk, dqw, dkw


# ---- sliding window ------------------------------------------------------------------------

def window_workspace_bytes(prob: Problem, window: int, sinks: int, which: int = 1) -> int:
    return int(lib().ra_window_workspace_bytes(prob.ptr, window, sinks, which))


def window_attn_fwd(q, k, v, prob: Problem, window: int, sinks: int = 0, out=None, lse=None,
                    workspace=None, stream=None):
    """Ring attention in which a query at position p sees the keys at k <= p with k > p -
    ``window`` or k < ``sinks`` -> (out, lse), shard-major. The workspace
    (``window_workspace_bytes(..., 0)``) is allocated when not given."""
    r, dev = prob.raw, q.get_device()
    made = []
    out = _made_like(q, made) if out is None else out
    if lse is None:
        made.append(lse := torch.empty(ops._lse_shape(prob), device=q.device, dtype=torch.float32))
    nq, nk = prob.rows * r.hq * r.head_dim, prob.rows * r.hkv * r.head_dim
    for t, n, name in ((q, nq, "q"), (k, nk, "k"), (v, nk, "v"), (out, nq, "out")):
        _token(t, n, name, prob, dev)
    _plain(lse, "lse", torch.float32, ops._lse_shape(prob), dev)
    workspace, size = _workspace(
        workspace, workspace is None and window_workspace_bytes(prob, window, sinks, 0), q, made)
    _launch(dev, stream, made, lambda s: lib().ra_window_attn_fwd(
        prob.ptr, window, sinks, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(workspace),
        size, s))
    return out, lse


def window_attn_bwd(dout, q, k, v, out, lse, prob: Problem, window: int, sinks: int = 0, dq=None,
                    dk=None, dv=None, workspace=None, stream=None):
    """Backward of ``window_attn_fwd`` -> (dq, dk, dv), shard-major, in the problem dtype."""
    r, dev = prob.raw, q.get_device()
    made = []
    dq = _made_like(q, made) if dq is None else dq
    dk = _made_like(k, made) if dk is None else dk
    dv = _made_like(v, made) if dv is None else dv
    nq, nk = prob.rows * r.hq * r.head_dim, prob.rows * r.hkv * r.head_dim
    for t, n, name in ((dout, nq, "dout"), (q, nq, "q"), (k, nk, "k"), (v, nk, "v"), (out, nq, "out"),
                       (dq, nq, "dq"), (dk, nk, "dk"), (dv, nk, "dv")):
        _token(t, n, name, prob, dev)
    _plain(lse, "lse", torch.float32, ops._lse_shape(prob), dev)
    workspace, size = _workspace(
        workspace, workspace is None and window_workspace_bytes(prob, window, sinks, 1), q, made)
    _launch(dev, stream, made, lambda s: lib().ra_window_attn_bwd(
        prob.ptr, window, sinks, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
        _ptr(workspace), size, s))
    return dq, dk, dv


# ---- the paged cache -----------------------------------------------------------------------

@dataclass
class PagedCache:
    """A paged key-value cache; ``raw`` is the C struct handed to the library. Keeps the
    tensors alive."""

    raw: RaPagedCache
    k_pages: torch.Tensor
    v_pages: torch.Tensor
    block_table: torch.Tensor

    def __post_init__(self):
        r = self.raw
        self.ptr = ctypes.byref(r)
        self.dtype, self.device_index = self.k_pages.dtype, self.k_pages.get_device()
        self.n_seqs, self.hkv, self.head_dim = r.n_seqs, r.hkv, r.head_dim


def make_cache(k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor) -> PagedCache:
    """A cache over k_pages and v_pages [n_pages, page_size, hkv, head_dim] (any strides with
    head_dim innermost, e.g. a transposed [n_pages, hkv, page_size, head_dim]; the same for
    both) and block_table [n_seqs, max_pages] (int32)."""
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype:
        raise ValueError("k_pages and v_pages must be [n_pages, page_size, hkv, head_dim] of one dtype")
    if k_pages.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"unsupported dtype {k_pages.dtype}")
    if block_table.dim() != 2 or block_table.dtype != torch.int32:
        raise ValueError("block_table must be an int32 tensor [n_seqs, max_pages]")
    devices = {t.device for t in (k_pages, v_pages, block_table)}
    if len(devices) != 1 or not k_pages.is_cuda:
        raise ValueError("k_pages, v_pages and block_table must be on one CUDA device")
    if k_pages.stride() != v_pages.stride() or (k_pages.shape[3] > 1 and k_pages.stride(3) != 1):
        raise ValueError("k_pages and v_pages must have the same strides, head_dim innermost")
    if block_table.shape[1] > 1 and block_table.stride(1) != 1:
        raise ValueError("the rows of block_table must be contiguous")
    raw = RaPagedCache()
    raw.dtype = RA_BF16 if k_pages.dtype == torch.bfloat16 else RA_F32
    raw.n_pages, raw.page_size, raw.hkv, raw.head_dim = k_pages.shape
    raw.n_seqs, raw.max_pages = block_table.shape
    raw.table_stride = max(block_table.stride(0), raw.max_pages) if raw.n_seqs <= 1 else block_table.stride(0)
    raw.page_stride, raw.slot_stride, raw.head_stride = k_pages.stride()[:3]
    raw.k_pages, raw.v_pages = k_pages.data_ptr(), v_pages.data_ptr()
    raw.block_table = block_table.data_ptr()
    return PagedCache(raw, k_pages, v_pages, block_table)


def kv_cache_append(q, k, v, cache: PagedCache, seq_lens, cu_new=None, q_weight=None, k_weight=None,
                    rope: Rope | AxisRope | None = None, eps: float = 1e-6, q_out=None, stream=None,
                    positions=None):
    """Put new tokens into the cache: norm and rotation of q and k as in ``qk_norm_rope_fwd``
    (None leaves them out), k and v to their pages -> q_out (None if q is None). seq_lens
    [n_seqs] int32 are the lengths with the new tokens. Without ``cu_new`` row b of q
    [n_seqs, hq, head_dim], k, v is the new token of sequence b (of length 0: idle, its row of
    q_out is 0); with it (int32 [n_seqs + 1], on the device) rows cu_new[b]:cu_new[b+1] are the
    last tokens of sequence b, and rows behind the last are left as they are. With an ``AxisRope``
    the rotation goes by ``positions`` (int32, [rows, n_axes])."""
    dt, dh, dev, hkv = cache.dtype, cache.head_dim, cache.device_index, cache.hkv
    n = k.shape[0] if k.dim() == 3 else k.shape[0] * k.shape[1]
    ks = _rows(k, "k", dt, n, hkv, dh, dev)
    vs = _rows(v, "v", dt, n, hkv, dh, dev)
    _weights(q_weight, k_weight, dt, dh, dev)
    _plain(seq_lens, "seq_lens", torch.int32, (cache.n_seqs,), dev)
    if cu_new is not None:
        _plain(cu_new, "cu_new", torch.int32, (cache.n_seqs + 1,), dev)
    hq, qs, made = 0, 0, []
    if q is not None:
        hq = q.shape[-2]
        qs = _rows(q, "q", dt, n, hq, dh, dev)
        q_out = _made_like(q, made) if q_out is None else _plain(q_out, "q_out", dt, q.shape, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    axes, ps = _positions(rope, positions, n, dev)
    rest = (eps, n, hq, _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(q_weight), _ptr(k_weight), _ptr(seq_lens),
            _ptr(cu_new), _ptr(q_out))
    if axes:
        _launch(dev, stream, made, lambda s: lib().ra_kv_cache_append_axes(cache.ptr, rope.ptr, _ptr(positions), ps,
                                                                           *rest, s))
    else:
        _launch(dev, stream, made, lambda s: lib().ra_kv_cache_append(cache.ptr, _rope_ptr(rope), *rest, s))
    return q_out


def paged_workspace_bytes(cache: PagedCache, hq: int) -> int:
    return int(lib().ra_paged_workspace_bytes(cache.ptr, hq))


def paged_attn_decode(q, cache: PagedCache, seq_lens, window: int = 0, sinks: int = 0,
                      scale: float | None = None, out=None, lse=None, workspace=None, stream=None,
                      shared: SharedPrefix | None = None):
    """Attention of the last token of every sequence over the cache -> (out, lse): q, out
    [n_seqs, hq, head_dim], lse [n_seqs, hq] float32 (natural log). With ``window`` > 0 only the
    last ``window`` and the first ``sinks`` of the seq_lens[b] keys are seen. A sequence of
    length 0 gets out = 0, lse = -inf. With ``shared`` the keys that groups of sequences have in
    common are read once for the group, as exactly as apart. The workspace (``paged_workspace_bytes``, with ``shared``
    ``paged_extend_workspace_bytes``) is allocated when not given."""
    if shared is not None:
        return paged_attn_extend(q, cache, seq_lens, None, shared, window, sinks, scale, out, lse, workspace, stream)
    dt, dev, n = cache.dtype, cache.device_index, cache.n_seqs
    if q.dim() != 3:
        raise ValueError("q must be [n_seqs, hq, head_dim]")
    shape = q.shape
    hq = shape[1]
    _plain(q, "q", dt, (n, hq, cache.head_dim), dev)
    _plain(seq_lens, "seq_lens", torch.int32, (n,), dev)
    made = []
    out = _made_like(q, made) if out is None else _plain(out, "out", dt, shape, dev)
    if lse is None:
        made.append(lse := torch.empty((n, hq), device=q.device, dtype=torch.float32))
    else:
        _plain(lse, "lse", torch.float32, (n, hq), dev)
    workspace, size = _workspace(workspace, workspace is None and paged_workspace_bytes(cache, hq), q, made)
    _launch(dev, stream, made, lambda s: lib().ra_paged_attn_decode(
        cache.ptr, hq, 0.0 if scale is None else scale, window, sinks, _ptr(q), _ptr(seq_lens), _ptr(out),
        _ptr(lse), _ptr(workspace), size, s))
    return out, lse


# ---- several new tokens, shared prefixes ---------------------------------------------------

@dataclass
class SharedPrefix:
    """Prefixes that groups of a cache's sequences have in common: the sequences cu_groups[g] ..
    cu_groups[g+1]-1 begin with the same prefix_lens[g] tokens, as a rule in the same pages. int32
    on the device, cu_groups [n_groups + 1], prefix_lens [n_groups]; their values are read when a
    call runs."""

    cu_groups: torch.Tensor
    prefix_lens: torch.Tensor

    def __post_init__(self):
        n = self.prefix_lens.numel()
        for t, name, size in ((self.cu_groups, "cu_groups", n + 1), (self.prefix_lens, "prefix_lens", n)):
            if t.dtype != torch.int32 or t.shape != (size,) or not t.is_contiguous() or not t.is_cuda:
                raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of {size} elements, got {t.dtype} "
                                 f"{tuple(t.shape)} on {t.device}")
        if self.cu_groups.device != self.prefix_lens.device:
            raise ValueError("cu_groups and prefix_lens must be on the same device")
        self.n_groups = n
        self.raw = RaSharedPrefix(n, self.cu_groups.data_ptr(), self.prefix_lens.data_ptr())
        self.ptr = ctypes.byref(self.raw)


def paged_extend_workspace_bytes(cache: PagedCache, n_tokens: int, hq: int, shared: SharedPrefix | None = None) -> int:
    n = 0 if shared is None else shared.n_groups
    return int(lib().ra_paged_extend_workspace_bytes(cache.ptr, n, n_tokens, hq))


def paged_attn_extend(q, cache: PagedCache, seq_lens, cu_new=None, shared: SharedPrefix | None = None,
                      window: int = 0, sinks: int = 0, scale: float | None = None, out=None, lse=None,
                      workspace=None, stream=None):
    """Causal attention of the last tokens of every sequence, which are in the cache already ->
    (out, lse): q, out [n_tokens, hq, head_dim], lse [n_tokens, hq] float32 (natural log). seq_lens
    [n_seqs] int32 are the lengths with the new tokens; rows cu_new[b]:cu_new[b+1] (int32
    [n_seqs + 1], on the device) are the last tokens of sequence b, other rows are left as they
    are. Without ``cu_new`` every sequence has one new token, or is idle (length 0: out = 0, lse =
    -inf). The row at position p sees the keys k <= p, with ``window`` > 0 those with k > p -
    window or k < sinks. With ``shared`` (not with a window) the keys that groups of sequences have
    in common are read once for the group where that saves work. In bf16 the weights of rows that are few
    are two bf16 numbers, of others one (include/ringattn.h has the rule). The workspace
    (``paged_extend_workspace_bytes``) is allocated when not given."""
    dt, dev = cache.dtype, cache.device_index
    if q.dim() != 3:
        raise ValueError("q must be [n_tokens, hq, head_dim]")
    shape = q.shape
    n, hq = shape[0], shape[1]
    _plain(q, "q", dt, (n, hq, cache.head_dim), dev)
    _plain(seq_lens, "seq_lens", torch.int32, (cache.n_seqs,), dev)
    if cu_new is not None:
        _plain(cu_new, "cu_new", torch.int32, (cache.n_seqs + 1,), dev)
    if shared is not None and shared.cu_groups.get_device() != dev:
        raise ValueError(f"shared must be on CUDA device {dev}")
    made = []
    out = _made_like(q, made) if out is None else _plain(out, "out", dt, shape, dev)
    if lse is None:
        made.append(lse := torch.empty((n, hq), device=q.device, dtype=torch.float32))
    else:
        _plain(lse, "lse", torch.float32, (n, hq), dev)
    workspace, size = _workspace(
        workspace, workspace is None and paged_extend_workspace_bytes(cache, n, hq, shared), q, made)
    _launch(dev, stream, made, lambda s: lib().ra_paged_attn_extend(
        cache.ptr, None if shared is None else shared.ptr, n, hq, 0.0 if scale is None else scale, window, sinks,
        _ptr(q), _ptr(seq_lens), _ptr(cu_new), _ptr(out), _ptr(lse), _ptr(workspace), size, s))
    return out, lse
