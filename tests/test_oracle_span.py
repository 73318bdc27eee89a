"""The span oracle against scalar code and differences."""

import math

import numpy as np
import pytest

from oracle.span import gather_pages, span_attention_bwd_ref, span_attention_ref, span_seen


def test_spans():
    seen = span_seen(4, begin=[0, 0, 2, 9], end=[4, -1, 4, 12], causal=True, window=2)
    assert seen.tolist() == [[True, False, False, False], [False] * 4, [False, False, True, False], [False] * 4]
    assert span_seen(2, causal=True, window=3, first=5, keys=8).tolist() == [
        [False, False, False, True, True, True, False, False], [False, False, False, False, True, True, True, False]]
    assert span_seen(3, window=2).tolist() == [[True, True, False], [True, True, True], [False, True, True]]


@pytest.mark.parametrize("cap,slope,first", [(0.0, 0.0, 0), (1.5, 0.0, 0), (0.0, 0.3, 2), (2.0, -0.1, 2)])
def test_one_row_at_a_time(cap, slope, first):
    g = np.random.default_rng(1)
    n, m, d = 5, 7, 4
    q, k, v = g.standard_normal((n, d)), g.standard_normal((m, d)), g.standard_normal((m, d))
    seen = span_seen(n, causal=True, window=4, first=first, keys=m)
    seen[3] = False
    o, lse, size, eo, el = span_attention_ref(q, k, v, 0.7, seen, cap, slope, first)
    for i in range(n):
        w = []
        for j in range(m):
            s = 0.7 * float(q[i] @ k[j])
            s = cap * math.tanh(s / cap) if cap else s
            w.append(math.exp(s - slope * abs(first + i - j)) if seen[i, j] else 0.0)
        total = sum(w)
        want = sum(x * v[j] for j, x in enumerate(w)) / total if total else np.zeros(d)
        np.testing.assert_allclose(o[i], want, rtol=1e-12, atol=1e-14)
        assert lse[i] == (pytest.approx(math.log(total), rel=1e-12) if total else -math.inf)
    assert (size >= np.abs(o) - 1e-15).all() and (eo >= 0).all() and (el >= 0).all()


@pytest.mark.parametrize("cap,slope", [(0.0, 0.0), (1.5, 0.0), (0.0, 0.3), (2.0, 0.1)])
def test_gradients_against_differences(cap, slope):
    g = np.random.default_rng(2)
    n, d = 6, 3
    x = [g.standard_normal((n, d)) for _ in range(3)]
    do = g.standard_normal((n, d))
    seen = span_seen(n, begin=[0, 0, 1, 1, 9, 0], causal=True, window=5)

    def f(y):
        return (span_attention_ref(*y, 0.6, seen, cap, slope)[0] * do).sum()

    o, lse = span_attention_ref(*x, 0.6, seen, cap, slope)[:2]
    grads, _, _ = span_attention_bwd_ref(*x, o, do, lse, 0.6, seen, cap, slope)
    for i in range(3):
        for at in np.ndindex(n, d):
            up, down = [y.copy() for y in x], [y.copy() for y in x]
            up[i][at] += 1e-6
            down[i][at] -= 1e-6
            assert grads[i][at] == pytest.approx((f(up) - f(down)) / 2e-6, rel=1e-6, abs=1e-8)


def test_pages():
    pages = np.arange(5 * 2 * 3, dtype=np.float64).reshape(5, 2, 3)
    got = gather_pages(pages, [3, -1, 0, 9], 5)
    assert got.tolist() == [*pages[3].tolist(), [0, 0, 0], [0, 0, 0], pages[0, 0].tolist()]
