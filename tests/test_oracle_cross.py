"""The cross attention, tree and rotation oracle against loops over its
definitions and against differences."""

import numpy as np
import pytest

from oracle import attention_bwd_ref, attention_fwd_ref
from oracle.cross import masked_attention_bwd_ref, masked_attention_ref, rope_bwd_ref, rope_ref, tree_visible


def rnd(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def test_agrees_with_the_square_oracle():
    q, k, v, do = (rnd(i, 9, 16) for i in range(4))
    for causal in (False, True):
        seen = np.tril(np.ones((9, 9), bool)) if causal else np.ones((9, 9), bool)
        o, lse, _ = masked_attention_ref(q, k, v, 0.3, seen)
        args = [x[None, None] for x in (q, k, v)]
        o_ref, lse_ref = attention_fwd_ref(*args, 0.3, causal)
        np.testing.assert_allclose(o, o_ref[0, 0], atol=1e-12)
        np.testing.assert_allclose(lse, lse_ref[0, 0], atol=1e-12)
        grads, _, _ = masked_attention_bwd_ref(q, k, v, o, do, lse, 0.3, seen)
        for g, r in zip(grads, attention_bwd_ref(*args, do[None, None], 0.3, causal)):
            np.testing.assert_allclose(g, r[0, 0], atol=1e-12)


def test_rows_that_see_nothing_and_nan_in_unseen_keys():
    q, k, v = rnd(1, 3, 8), rnd(2, 5, 8), rnd(3, 5, 8)
    seen = np.zeros((3, 5), bool)
    seen[0, :2] = seen[2, 1] = True
    k[3:], v[3:] = np.nan, np.inf
    o, lse, _ = masked_attention_ref(q, k, v, 1.0, seen)
    assert (o[1] == 0).all() and np.isneginf(lse[1])
    np.testing.assert_allclose(o[2], v[1])
    assert np.isfinite(o).all()


def test_attention_gradients_against_differences():
    q, k, v, do = rnd(1, 4, 6), rnd(2, 7, 6), rnd(3, 7, 6), rnd(4, 4, 6)
    seen = np.random.default_rng(5).random((4, 7)) < 0.6
    seen[1] = False
    o, lse, _ = masked_attention_ref(q, k, v, 0.5, seen)
    grads, _, _ = masked_attention_bwd_ref(q, k, v, o, do, lse, 0.5, seen)
    h = 1e-5
    for i, g in enumerate(grads):
        u = rnd(10 + i, *g.shape)
        f = []
        for sign in (1, -1):
            x = [q, k, v]
            x[i] = x[i] + sign * h * u
            f.append((masked_attention_ref(*x, 0.5, seen)[0] * do).sum())
        assert abs((f[0] - f[1]) / (2 * h) - (g * u).sum()) < 1e-8


def test_tree_visibility():
    seen = tree_visible(2, 3, 4, 6, [0b001, 0b011, 0b101, 0b1111])
    assert seen.astype(int).tolist() == [[1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 0, 0], [1, 1, 1, 0, 1, 0], [1, 1, 1, 1, 1, 0]]
    assert tree_visible(1, 2, 2, 2).astype(int).tolist() == [[1, 1], [1, 1]]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("eps", [None, 1e-3])
def test_rotation_and_its_gradients(interleaved, eps):
    x, w, dy = rnd(1, 2, 5, 8), rnd(2, 8), rnd(3, 2, 5, 8)
    freq, pos = np.array([0.7, 0.1, 0.01]), np.array([0, 1, 5, 900, 7])
    y = rope_ref(x, w, freq, pos, eps, 1.5, interleaved)
    for t in range(5):
        for i in range(3):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 3)
            u = x[1, t] / (1.0 if eps is None else np.sqrt((x[1, t] ** 2).mean() + eps)) * (1.0 if eps is None else w)
            z = 1.5 * (u[a] + 1j * u[b]) * np.exp(1j * pos[t] * freq[i])
            np.testing.assert_allclose([y[1, t, a], y[1, t, b]], [z.real, z.imag], atol=1e-12)
    dx, dw = rope_bwd_ref(x, w, freq, pos, dy, eps, 1.5, interleaved)
    h, u, uw = 1e-6, rnd(4, *x.shape), rnd(5, 8)

    def f(x, w):
        return (rope_ref(x, w, freq, pos, eps, 1.5, interleaved) * dy).sum()

    assert abs((f(x + h * u, w) - f(x - h * u, w)) / (2 * h) - (dx * u).sum()) < 1e-7
    if eps is None:
        assert dw is None
    else:
        assert abs((f(x, w + h * uw) - f(x, w - h * uw)) / (2 * h) - (dw * uw).sum()) < 1e-7
