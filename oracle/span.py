"""fp64 oracle of attention to spans of keys with capped scores and a distance bias,
and of caches in pages.  numpy only; shares no code with the kernels.
"""

from __future__ import annotations

import numpy as np


def span_seen(n: int, begin=None, end=None, causal=False, window=0, first=0, keys=None) -> np.ndarray:
    """[n, keys]: the keys that each query sees.  Query i is at position first + i;
    begin, end: n integers or None (0 and keys); keys: n by default."""
    keys = n if keys is None else keys
    pos = first + np.arange(n)[:, None]
    j = np.arange(keys)[None]
    seen = np.ones((n, keys), dtype=bool)
    if begin is not None:
        seen &= j >= np.asarray(begin, dtype=np.int64)[:, None]
    if end is not None:
        seen &= j < np.asarray(end, dtype=np.int64)[:, None]
    if causal:
        seen &= j <= pos
    if window:
        seen &= np.abs(pos - j) < window
    return seen


def span_scores(q, k, scale, cap=0.0, slope=0.0, first=0):
    """(s, 1 - tanh^2, E): scores of q [n,d] and k [m,d], the factor of their gradient,
    and a bound on what fp32 makes of them: (d + 2) 2^-24 of the product's terms, a tanh
    that is off by 2^-21, and 2^-22 of what is added up and of the exponential."""
    q, k = q.astype(np.float64), k.astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        s = scale * (q @ k.T)
        err = (q.shape[1] + 2) * 2.0 ** -24 * scale * (np.abs(q) @ np.abs(k).T)
    bent = np.ones_like(s)
    if cap:
        t = np.tanh(s / cap)
        bent, s, err = 1.0 - t * t, cap * t, err + cap * 2.0 ** -21
    far = np.abs(first + np.arange(q.shape[0])[:, None] - np.arange(k.shape[0])[None])
    s = s - slope * far
    return s, bent, err + 2.0 ** -22 * (1.0 + np.abs(s) + 2 * abs(slope) * far)


def span_attention_ref(q, k, v, scale, seen, cap=0.0, slope=0.0, first=0):
    """One head: (O, LSE, A, EO, EL): A = sum_j P_ij |v_j|; EO, EL bound what the scores'
    errors do to O and LSE, sum_j P_ij E_ij (|v_j| + |O_i|) and sum_j P_ij E_ij.  Rows
    that see nothing give O = 0 and LSE = -inf; keys that no row sees have no effect."""
    used = seen.any(0)
    k, v = (np.where(used[:, None], x, 0).astype(np.float64) for x in (k, v))
    s, _, err = span_scores(q, k, scale, cap, slope, first)
    s = np.where(seen, s, -np.inf)
    m = s.max(1, initial=-np.inf)
    m = np.where(np.isneginf(m), 0.0, m)
    p = np.exp(s - m[:, None])
    total = p.sum(1)
    p = p / np.where(total == 0, 1.0, total)[:, None]
    o = p @ v
    pe = p * np.where(seen, err, 0.0)
    with np.errstate(divide="ignore"):
        return o, m + np.log(total), p @ np.abs(v), pe @ np.abs(v) + pe.sum(1)[:, None] * np.abs(o), pe.sum(1)


def span_attention_bwd_ref(q, k, v, o, do, lse, scale, seen, cap=0.0, slope=0.0):
    """Gradients of one head from the O and LSE at hand: (dq, dk, dv), the sizes that the
    rounding of P and dS scales with, and the sizes of fp32's errors (of the scores, and
    2e-4 of dS = P (dP - delta)'s terms)."""
    q, k, v, o, do, lse = (np.asarray(x, dtype=np.float64) for x in (q, k, v, o, do, lse))
    s, bent, err = span_scores(q, k, scale, cap, slope)
    live = seen & ~np.isneginf(lse)[:, None]
    p = np.where(live, np.exp(np.where(live, s - np.where(np.isneginf(lse), 0.0, lse)[:, None], 0.0)), 0.0)
    dp, delta = do @ v.T, (do * o).sum(1)
    ds = p * (dp - delta[:, None]) * bent
    off = np.abs(ds) * err + 2e-4 * p * (np.abs(do) @ np.abs(v).T + (np.abs(do) * np.abs(o)).sum(1)[:, None])
    grads = scale * (ds @ k), scale * (ds.T @ q), p.T @ do
    halves = scale * (np.abs(ds) @ np.abs(k)), scale * (np.abs(ds).T @ np.abs(q)), p.T @ np.abs(do)
    fp32 = scale * (off @ np.abs(k)), scale * (off.T @ np.abs(q)), (p * (err + 2e-4)).T @ np.abs(do)
    return grads, halves, fp32


def gather_pages(pages, table, tokens: int):
    """[tokens, d]: rows 0 .. tokens-1 of one request and head; pages [count, page_size, d], table the request's
    page numbers.  Numbers outside the pool are pages of zeros."""
    size = pages.shape[1]
    out = np.zeros((tokens, pages.shape[2]), dtype=np.float64)
    for first in range(0, tokens, size):
        page = int(table[first // size])
        if 0 <= page < pages.shape[0]:
            n = min(size, tokens - first)
            out[first:first + n] = pages[page, :n]
    return out
