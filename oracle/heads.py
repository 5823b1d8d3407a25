"""Head norms with rotation, attention over a paged cache and windowed attention, in float64.

The definitions, literally and for small sizes: a rotation as a multiplication by complex
numbers, a cache read token by token through its table, a window as a dense boolean mask.
"""
from __future__ import annotations

import numpy as np


def phases(pos, inv_freq):
    """exp(i pos inv_freq), [tokens, pairs]."""
    return np.exp(1j * np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None, :])


def turn(x, z, interleaved):
    """The first 2 * pairs elements of every head of x [tokens, heads, dh], read as complex
    numbers, multiplied by z [tokens, pairs]."""
    y, rd = np.array(x, np.float64), 2 * z.shape[1]
    a, b = (slice(0, rd, 2), slice(1, rd, 2)) if interleaved else (slice(0, rd // 2), slice(rd // 2, rd))
    c = (y[..., a] + 1j * y[..., b]) * z[:, None, :]
    y[..., a], y[..., b] = c.real, c.imag
    return y


def norm_rope_fwd(x, w, z, eps, interleaved=False):
    """x [tokens, heads, dh] -> y; w None: no norm, z None: no rotation."""
    y = np.asarray(x, np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w
    return y if z is None else turn(y, z, interleaved)


def norm_rope_bwd(dy, x, w, z, eps, interleaved=False):
    """(dx, dw) of norm_rope_fwd; dw None without a norm."""
    g = np.asarray(dy, np.float64)
    if z is not None:
        g = turn(g, z.conj(), interleaved)
    if w is None:
        return g, None
    x = np.asarray(x, np.float64)
    ms = (x * x).mean(-1, keepdims=True) + eps
    dw = (g * x / np.sqrt(ms)).sum((0, 1))
    h = g * w
    return h / np.sqrt(ms) - x * (h * x).mean(-1, keepdims=True) / ms ** 1.5, dw


def gather(pages, table_row, n):
    """The first n tokens of a sequence from pages [n_pages, page_size, heads, dh]."""
    size = pages.shape[1]
    return np.stack([pages[table_row[t // size], t % size] for t in range(n)]) if n else \
        np.zeros((0,) + pages.shape[2:])


def seen(n_q, n_k, window, sinks):
    """Mask [n_q, n_k] of the last n_q of n_k tokens: causal, and with a window only the last
    ``window`` keys up to the query's own and the first ``sinks``."""
    p = np.arange(n_k - n_q, n_k)[:, None]
    j = np.arange(n_k)[None, :]
    ok = j <= p
    if window:
        ok &= (j > p - window) | (j < sinks)
    return ok


def masked_fwd(q, k, v, ok, scale):
    """Attention of q [nq, hq, dh] to k, v [nk, hkv, dh] under a mask -> out, lse [hq, nq]; a
    query that sees nothing gets 0 and -inf."""
    nq, hq, dh = q.shape
    grp = hq // k.shape[1]
    out, lse = np.zeros((nq, hq, dh)), np.full((hq, nq), -np.inf)
    for h in range(hq):
        s = np.where(ok, scale * q[:, h] @ k[:, h // grp].T, -np.inf)
        m = s.max(-1, initial=-np.inf, keepdims=True)
        e = np.exp(s - np.where(np.isfinite(m), m, 0.0))
        l = e.sum(-1, keepdims=True)
        with np.errstate(divide="ignore"):
            lse[h] = (np.where(np.isfinite(m), m, 0.0) + np.log(l))[:, 0]
        out[:, h] = (e / np.where(l > 0, l, 1.0)) @ v[:, h // grp]
    return out, lse


def masked_bwd(q, k, v, do, ok, scale):
    """Textbook gradient of masked_fwd -> dq, dk, dv."""
    grp = q.shape[1] // k.shape[1]
    out, lse = masked_fwd(q, k, v, ok, scale)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for h in range(q.shape[1]):
        g = h // grp
        s = np.where(ok, scale * q[:, h] @ k[:, g].T, -np.inf)
        p = np.exp(s - np.where(np.isfinite(lse[h]), lse[h], 0.0)[:, None])
        dp = do[:, h] @ v[:, g].T
        ds = p * (dp - (do[:, h] * out[:, h]).sum(-1, keepdims=True))
        dq[:, h] = scale * ds @ k[:, g]
        dk[:, g] += scale * ds.T @ q[:, h]
        dv[:, g] += p.T @ do[:, h]
    return dq, dk, dv
