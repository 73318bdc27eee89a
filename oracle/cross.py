"""fp64 oracle of attention with keys of another length, of drafted trees over a
cache, and of the head norm and rotation, with their gradients.  numpy only;
shares no code with the kernels.
"""

from __future__ import annotations

import numpy as np


def tree_visible(length: int, drafts: int, T: int, C: int, masks=None) -> np.ndarray:
    """[T, C]: the cache rows that each new token sees.  masks: T ints, bit t of
    masks[n] says whether token n sees token t (None: t <= n)."""
    seen = np.zeros((T, C), dtype=bool)
    seen[:, :length] = True
    for n in range(T):
        for t in range(min(drafts, C - length)):
            seen[n, length + t] = t <= n if masks is None else bool((int(masks[n]) >> t) & 1)
    return seen


def masked_attention_ref(q, k, v, scale, seen):
    """One head: q [n,d], k, v [m,d], seen [n,m].  Returns (O, LSE, A) with
    A = sum_j P_ij |v_j|, the size that rounding errors of P scale with.
    Rows that see nothing give O = 0 and LSE = -inf; what unseen rows of k and v
    hold has no effect."""
    used = seen.any(0)
    q, k, v = q.astype(np.float64), np.where(used[:, None], k, 0).astype(np.float64), np.where(used[:, None], v, 0).astype(np.float64)
    s = np.where(seen, scale * (q @ k.T), -np.inf)
    m = s.max(1, initial=-np.inf)
    m = np.where(np.isneginf(m), 0.0, m)
    p = np.exp(s - m[:, None])
    l = p.sum(1)
    p = p / np.where(l == 0, 1.0, l)[:, None]
    with np.errstate(divide="ignore"):
        return p @ v, m + np.log(l), p @ np.abs(v)


def masked_attention_bwd_ref(q, k, v, o, do, lse, scale, seen):
    """Gradients of one head from the O and LSE at hand: (dq, dk, dv), and for
    each the size its rounding errors scale with (see grad_bounds)."""
    used = seen.any(0)
    q, o, do, lse = (np.asarray(x, dtype=np.float64) for x in (q, o, do, lse))
    k, v = (np.where(used[:, None], x, 0).astype(np.float64) for x in (k, v))
    p = np.where(seen, np.exp(np.where(seen, scale * (q @ k.T) - lse[:, None], 0.0)), 0.0)
    dp, delta = do @ v.T, (do * o).sum(1)
    ds = p * (dp - delta[:, None])
    # what fp32 arithmetic of dS = P (dP - delta) is relative to
    dp_size = p * (np.abs(do) @ np.abs(v).T + (np.abs(do) * np.abs(o)).sum(1)[:, None])
    grads = scale * (ds @ k), scale * (ds.T @ q), p.T @ do
    halves = scale * (np.abs(ds) @ np.abs(k)), scale * (np.abs(ds).T @ np.abs(q)), p.T @ np.abs(do)
    fp32 = scale * (dp_size @ np.abs(k)), scale * (dp_size.T @ np.abs(q)), p.T @ np.abs(do)
    return grads, halves, fp32


def rope_ref(x, weight, freq, pos, eps=None, factor=1.0, interleaved=False):
    """x [..., n, d] (n tokens), pos [n]: head norm (with eps) and rotation."""
    x = x.astype(np.float64)
    if eps is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            x = x * weight.astype(np.float64)
    half = len(freq)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    angle = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(freq, dtype=np.float64)
    c, s = factor * np.cos(angle), factor * np.sin(angle)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def rope_bwd_ref(x, weight, freq, pos, dy, eps=None, factor=1.0, interleaved=False):
    """(dx, dweight) of rope_ref; dweight summed over everything but d (None without eps)."""
    g = rope_ref(dy, None, -np.asarray(freq, dtype=np.float64), pos, None, factor, interleaved)
    if eps is None:
        return g, None
    x = x.astype(np.float64)
    d = x.shape[-1]
    inv = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    unit = x * inv
    dw = (g * unit).reshape(-1, d).sum(0)
    if weight is not None:
        g = g * weight.astype(np.float64)
    return inv * (g - unit * (g * unit).mean(-1, keepdims=True)), dw
