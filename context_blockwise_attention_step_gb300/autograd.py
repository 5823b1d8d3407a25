"""Autograd wrappers and a drop-in attention module over the ring-attention C ABI.

The ring-flash-attn package card ("quickstart") shows the adapter use of ring attention:
a model keeps its projections and swaps its attention call for the ring one, and the
nanotron how-to page ("Integrating with MultiHeadAttention") selects ring attention by
name in its attention registry. Here the same is done on one GPU: ``ring_attention`` is a
differentiable call (forward = ``ra_ring_attn_fwd``, backward = ``ra_ring_attn_bwd`` against
the saved out and lse), ``shard`` / ``unshard`` move token tensors between natural and
shard-major order with their inverse permutation as gradient, ``qk_norm_rope`` is the head norm
and rotation before it, and ``RingSelfAttention`` is a multi-head (GQA) self-attention layer with
random weights that uses them, with a serving form over a paged key-value cache.

Gradients are of first order: a second derivative through the attention or the head norm raises (the
permutations have theirs).

A backward captured into a CUDA graph wants the gradients by ``torch.autograd.grad``, or no other
graph of the same parameters alive: accumulating into ``.grad`` would run on the stream of the
first graph, outside the capture.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import heads, ops


class _RingAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, prob, window, sinks):
        if window:
            out, lse = heads.window_attn_fwd(q, k, v, prob, window, sinks)
        else:
            out, lse = ops.ring_attn_fwd(q, k, v, prob)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.prob, ctx.window, ctx.sinks = prob, window, sinks
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, _dlse):
        q, k, v, out, lse = ctx.saved_tensors
        if ctx.window:
            grads = heads.window_attn_bwd(dout.contiguous(), q, k, v, out, lse, ctx.prob, ctx.window, ctx.sinks)
        else:
            grads = ops.ring_attn_bwd(dout.contiguous(), q, k, v, out, lse, ctx.prob)
        return *grads, None, None, None


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, prob, rope, eps, positions):
        # without a norm the backward does not look at q and k
        ctx.save_for_backward(positions, *((q, k, q_weight, k_weight) if q_weight is not None else ()))
        ctx.prob, ctx.rope, ctx.eps = prob, rope, eps
        return heads.qk_norm_rope_fwd(q, k, prob, q_weight=q_weight, k_weight=k_weight, rope=rope, eps=eps,
                                      positions=positions)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        dq_out, dk_out = dq_out.contiguous(), dk_out.contiguous()
        positions, *saved = ctx.saved_tensors
        q, k, q_weight, k_weight = saved or (dq_out, dk_out, None, None)
        dq, dk, dqw, dkw = heads.qk_norm_rope_bwd(dq_out, dk_out, q, k, ctx.prob, q_weight=q_weight,
                                                  k_weight=k_weight, rope=ctx.rope, eps=ctx.eps, positions=positions)
        if dqw is not None:  # float32 sums, rounded once to the parameter's type
            dqw, dkw = dqw.to(q_weight.dtype), dkw.to(k_weight.dtype)
        return dq, dk, dqw, dkw, None, None, None, None


class _Shard(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, prob, direction):
        ctx.prob = prob
        ctx.direction = direction
        x = x.contiguous()
        return ops.shard_tokens(x, prob) if direction == 0 else ops.unshard_tokens(x, prob)

    @staticmethod
    def backward(ctx, g):
        return _Shard.apply(g, ctx.prob, 1 - ctx.direction), None, None


def ring_attention(q, k, v, prob: ops.Problem, window: int = 0, sinks: int = 0):
    """Differentiable ring attention on shard-major q, k, v; returns (out, lse). With ``window``
    > 0 a query sees its last ``window`` keys and the first ``sinks`` of the sequence."""
    if window < 0 or (sinks and not window):
        raise ValueError("sinks go with a window >= 1")
    return _RingAttention.apply(q, k, v, prob, window, sinks)


def qk_norm_rope(q, k, prob: ops.Problem, q_weight=None, k_weight=None,
                 rope: heads.Rope | heads.AxisRope | None = None, eps: float = 1e-6, positions=None):
    """Differentiable per-head norm and rotation by position of shard-major q and k (with an
    ``AxisRope`` by ``positions``, shard-major too)."""
    return _QkNormRope.apply(q, k, q_weight, k_weight, prob, rope, eps, positions)


def shard(x, prob: ops.Problem):
    """Natural -> shard-major order (gradient: the inverse permutation)."""
    return _Shard.apply(x, prob, 0)


def unshard(x, prob: ops.Problem):
    """Shard-major -> natural order (gradient: the inverse permutation)."""
    return _Shard.apply(x, prob, 1)


class RingSelfAttention(torch.nn.Module):
    """Self-attention with ring attention as its attention call.

    x [B, S, hidden] (natural order) -> y [B, S, hidden]. Query / key / value / output
    projections are ordinary linear layers (random initialisation, no bias); the attention
    between them runs through the library with D virtual ring shards in the chosen layout.
    With ``shard_major=True`` x and y are already shard-major (a model that shards its
    tokens once at the input keeps them so through every token-wise layer).

    ``qk_norm`` adds a norm of every query and key head (weights of head_dim), ``rope`` a rotation
    by position, ``window`` and ``sinks`` a sliding window with always visible first tokens. With an
    ``AxisRope`` every call takes the tokens' ``positions`` (int32, x's leading shape and n_axes).
    ``prefill``, ``extend`` and ``decode`` are the layer's serving form over a paged key-value cache.
    """

    def __init__(self, hidden: int, hq: int, hkv: int, head_dim: int, *, D: int,
                 layout: str = "zigzag", causal: bool = True, shard_major: bool = False,
                 device=None, dtype=torch.bfloat16, seed: int = 0, qk_norm: bool = False,
                 rope: heads.Rope | heads.AxisRope | None = None, window: int = 0, sinks: int = 0,
                 eps: float = 1e-6):
        super().__init__()
        if hq % hkv:
            raise ValueError("hq must be a multiple of hkv")
        if window < 0 or (sinks and not window):
            raise ValueError("sinks go with a window >= 1")
        self.rope, self.window, self.sinks, self.eps = rope, window, sinks, eps
        self.hq, self.hkv, self.head_dim = hq, hkv, head_dim
        self.D, self.layout, self.causal, self.shard_major = D, layout, causal, shard_major
        g = torch.Generator().manual_seed(seed)

        def lin(n_out, n_in):
            w = torch.randn(n_out, n_in, generator=g) / math.sqrt(n_in)
            return torch.nn.Parameter(w.to(device=device, dtype=dtype))

        self.wq = lin(hq * head_dim, hidden)
        self.wk = lin(hkv * head_dim, hidden)
        self.wv = lin(hkv * head_dim, hidden)
        self.wo = lin(hidden, hq * head_dim)
        self.q_norm = self.k_norm = None
        if qk_norm:
            self.q_norm = torch.nn.Parameter(torch.ones(head_dim, device=device, dtype=dtype))
            self.k_norm = torch.nn.Parameter(torch.ones(head_dim, device=device, dtype=dtype))

    def problem(self, batch: int, seqlen: int) -> ops.Problem:
        return ops.make_problem(dtype=self.wq.dtype, layout=self.layout, causal=self.causal,
                                D=self.D, hq=self.hq, hkv=self.hkv, head_dim=self.head_dim,
                                batch=batch, seqlen=seqlen)

    def _qkv(self, x):
        lead = x.shape[:-1]
        return ((x @ self.wq.t()).view(*lead, self.hq, self.head_dim),
                (x @ self.wk.t()).view(*lead, self.hkv, self.head_dim),
                (x @ self.wv.t()).view(*lead, self.hkv, self.head_dim))

    def _attend(self, q, k, v, prob, positions):
        """Norm, rotation and attention of shard-major q, k, v -> (out, the k that was attended to)."""
        if self.q_norm is not None or self.rope is not None or positions is not None:
            q, k = qk_norm_rope(q, k, prob, self.q_norm, self.k_norm, self.rope, self.eps, positions)
        out, _ = ring_attention(q.contiguous(), k.contiguous(), v.contiguous(), prob, self.window, self.sinks)
        return out, k

    def forward(self, x, positions=None):
        b, s, _ = x.shape
        prob = self.problem(b, s)
        if positions is not None and positions.device != x.device:
            raise ValueError(f"positions must be on {x.device}, where x is, got {positions.device}")
        q, k, v = self._qkv(x)
        if not self.shard_major:
            q, k, v = shard(q, prob), shard(k, prob), shard(v, prob)
            if positions is not None:
                positions = ops.shard_tokens(positions.contiguous(), prob)
        out, _ = self._attend(q, k, v, prob, positions)
        if not self.shard_major:
            out = unshard(out, prob)
        return out.reshape(b, s, self.hq * self.head_dim) @ self.wo.t()

    @torch.no_grad()
    def prefill(self, x, cache: heads.PagedCache, cu_seqlens, positions=None):
        """The prompts of the cache's sequences, packed [T, hidden] in natural order with host
        offsets ``cu_seqlens`` [n_seqs + 1]: y [T, hidden], and their keys and values in the cache
        from its first place on."""
        if not self.causal:
            raise ValueError("a cache wants causal attention")
        prob = ops.make_problem(dtype=self.wq.dtype, layout="basic", causal=True, D=1, hq=self.hq,
                                hkv=self.hkv, head_dim=self.head_dim, cu_seqlens=cu_seqlens)
        q, k, v = self._qkv(x)
        out, k = self._attend(q, k, v, prob, positions)
        cu = torch.from_numpy(prob.cu_host).to(x.device)
        heads.kv_cache_append(None, k, v, cache, cu[1:] - cu[:-1], cu_new=cu)
        return out.reshape(x.shape[0], self.hq * self.head_dim) @ self.wo.t()

    def _append(self, x, cache, seq_lens, cu_new, positions):
        """New tokens x into the cache -> their queries."""
        if not self.causal:
            raise ValueError("a cache wants causal attention")
        q, k, v = self._qkv(x)
        return heads.kv_cache_append(q, k, v, cache, seq_lens, cu_new=cu_new, q_weight=self.q_norm,
                                     k_weight=self.k_norm, rope=self.rope, eps=self.eps, positions=positions)

    @torch.no_grad()
    def extend(self, x, cache: heads.PagedCache, seq_lens, cu_new, positions=None,
               shared: heads.SharedPrefix | None = None, workspace=None):
        """Several new tokens of every sequence after those in the cache, packed x [T, hidden] -> y
        [T, hidden]: rows cu_new[b]:cu_new[b+1] (int32 [n_seqs + 1], on the device; from 0 to T) are the
        last of the seq_lens[b] tokens that sequence b has with them. ``shared`` tells of prefixes
        that sequences have in common (their keys are in the cache already); a layer with a window
        reads every sequence's own."""
        q = self._append(x, cache, seq_lens, cu_new, positions)
        out, _ = heads.paged_attn_extend(q, cache, seq_lens, cu_new, shared=None if self.window else shared,
                                         window=self.window, sinks=self.sinks, workspace=workspace)
        return out.view(x.shape[0], self.hq * self.head_dim) @ self.wo.t()

    @torch.no_grad()
    def decode(self, x, cache: heads.PagedCache, seq_lens, workspace=None, positions=None,
               shared: heads.SharedPrefix | None = None):
        """One new token of every sequence, x [n_seqs, hidden] -> y [n_seqs, hidden]. seq_lens
        [n_seqs] (int32, on the device) are the lengths with the new tokens; a sequence of length
        0 is idle, and its row of y is 0. ``shared`` as for ``extend``."""
        q = self._append(x, cache, seq_lens, None, positions)
        out, _ = heads.paged_attn_decode(q, cache, seq_lens, window=self.window, sinks=self.sinks,
                                         workspace=workspace, shared=None if self.window else shared)
        return out.view(x.shape[0], self.hq * self.head_dim) @ self.wo.t()
