"""Attention to spans of keys (fa_span_fwd, fa_span_bwd) against the fp64 oracle.

Bounds, elementwise.  H = 2^-8 is the half step of bf16; E bounds the error of a
score in fp32 (oracle.span.span_scores).
  O    each P is rounded to bf16 before it meets V and O once at the end, and the
       normaliser differs from the sum of the rounded P by at most H of it:
       H (A + 2 |O|) with A = sum_j P_j |v_j|; scores that are off by E move O by
       sum_j P_j E_j (|v_j| + |O|); fp32 exponentials and sums add at most 1e-4 A.
  LSE  sum_j P_j E_j, 1e-4 for the sums, and fp32's 2^-22 |LSE|.
  dV   H (sum_i P |dO| + |dV|) + sum_i P (E + 2e-4) |dO|
  dQ   H (scale sum_j |dS| |k| + |dQ|) + scale sum_j e |k| for the rounding of dS
       and of dQ, with e = |dS| E + 2e-4 P (|dO| |v| + |dO o|) for fp32's errors;
  dK   the same with q.  Sums over a group's heads add up.
"""

import math

import numpy as np
import pytest
import torch

from exact_tiled_attention_08_gb300 import fa
from oracle.span import span_attention_bwd_ref, span_attention_ref, span_seen

pytestmark = pytest.mark.gpu

H2 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_tiled_attention_08_gb300.build import build_library

    build_library()
    fa.load_library()
    assert torch.cuda.is_available()


def randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).bfloat16()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def heads_of(B, H):
    """(b, h) pairs to check: all of them, or a spread of eight."""
    every = [(b, h) for b in range(B) for h in range(H)]
    return every if len(every) <= 8 else [every[i * (len(every) - 1) // 7] for i in range(8)]


def masks(kind, B, N, seed):
    """key_begin, key_end (int32 [B, N] or None) and causal."""
    g = np.random.default_rng(seed)
    begin, end = np.zeros((B, N), np.int32), np.full((B, N), N, np.int32)
    if kind in ("full", "causal"):
        return None, None, kind == "causal"
    if kind == "random":  # any two numbers, some outside the keys, some in the wrong order
        return (torch.from_numpy(g.integers(-N - 3, N + 3, (B, N)).astype(np.int32)),
                torch.from_numpy(g.integers(-2, 2 * N + 3, (B, N)).astype(np.int32)), False)
    if kind == "prefix":
        for b in range(B):
            end[b] = np.maximum(np.arange(N) + 1, g.integers(0, N + 1))
        return None, torch.from_numpy(end), False
    end[:] = 0
    for b in range(B):  # documents, and padding behind the last
        at = 0
        while at < N - N // 8:
            n = int(g.integers(1, max(2, N // 3)))
            n = min(n, N - N // 8 - at)
            begin[b, at:at + n], end[b, at:at + n] = at, at + n
            at += n
    return torch.from_numpy(begin), torch.from_numpy(end), kind == "docs"


def inputs(B, H, Hkv, N, d, cap, seed):
    q, k, v, do = randn(seed, B, H, N, d), randn(seed + 1, B, Hkv, N, d), randn(seed + 2, B, Hkv, N, d), \
        randn(seed + 3, B, H, N, d)
    return (q * 4 if cap else q), k, v, do


def slopes_of(H, on):
    return 2.0 ** (-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H) if on else None


def seen_of(begin, end, causal, window, b, N):
    return span_seen(N, None if begin is None else begin[b].numpy(), None if end is None else end[b].numpy(), causal,
                     window)


def check_rows(o, lse, ref, what):
    ro, rl, size, eo, el = ref
    err = np.abs(o - ro)
    bound = H2 * (size + 2 * np.abs(ro)) + 1e-4 * size + eo
    assert (err <= bound).all(), (what, "o", (err - bound).max(), np.argwhere(~(err <= bound))[:4])
    dead = np.isneginf(rl)
    assert np.isneginf(lse[dead]).all() and (o[dead] == 0).all(), what
    err = np.abs(lse[~dead] - rl[~dead])
    assert (err <= 1e-4 + el[~dead] + 2.0 ** -22 * np.abs(rl[~dead])).all(), (what, "lse", err.max())


def check_fwd(q, k, v, o, lse, scale, begin, end, causal, window, cap, slopes):
    B, H, N, _ = q.shape
    G = H // k.shape[1]
    for b, h in heads_of(B, H):
        ref = span_attention_ref(host(q[b, h]), host(k[b, h // G]), host(v[b, h // G]), scale,
                                 seen_of(begin, end, causal, window, b, N), cap,
                                 0.0 if slopes is None else float(slopes[h]))
        check_rows(host(o[b, h]), host(lse[b, h]), ref, (b, h))


def check_bwd(q, k, v, o, do, lse, grads, scale, begin, end, causal, window, cap, slopes):
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    for b, j in heads_of(B, Hkv):
        seen = seen_of(begin, end, causal, window, b, N)
        sums = [np.zeros((3, N, d)) for _ in range(2)]
        for h in range(j * G, (j + 1) * G):
            g, half, fp32 = span_attention_bwd_ref(*(host(x) for x in (q[b, h], k[b, j], v[b, j], o[b, h], do[b, h],
                                                                       lse[b, h])), scale, seen, cap,
                                                   0.0 if slopes is None else float(slopes[h]))
            err = np.abs(host(grads[0][b, h]) - g[0])
            bound = H2 * (half[0] + np.abs(g[0])) + fp32[0] + 1e-30
            assert (err <= bound).all(), (b, h, "dq", (err - bound).max(), err.max())
            for i in (0, 1):
                sums[i] += np.stack([g[1 + i], half[1 + i], fp32[1 + i]])
        for name, got, (g, half, fp32) in (("dk", grads[1], sums[0]), ("dv", grads[2], sums[1])):
            err = np.abs(host(got[b, j]) - g)
            bound = H2 * (half + np.abs(g)) + fp32 + 1e-30
            assert (err <= bound).all(), (b, j, name, (err - bound).max(), err.max())


CASES = [
    # B, H, Hkv, N, mask, window, cap, slopes
    (1, 1, 1, 1, "full", 0, 0.0, False),
    (2, 4, 2, 1, "causal", 1, 30.0, True),
    (1, 2, 1, 3, "causal", 0, 0.0, True),
    (2, 2, 1, 77, "docs", 0, 20.0, False),
    (1, 2, 2, 127, "random", 0, 0.0, False),
    (1, 2, 2, 128, "causal", 0, 0.0, False),
    (2, 6, 2, 129, "prefix", 0, 0.0, True),
    (1, 4, 1, 255, "docs_full", 0, 50.0, True),
    (1, 4, 4, 256, "causal", 100, 0.0, False),
    (2, 8, 2, 257, "random", 60, 30.0, True),
    (3, 4, 4, 333, "docs", 0, 0.0, False),
    (1, 8, 2, 500, "full", 33, 0.0, True),
    (2, 5, 1, 513, "docs", 128, 0.0, False),
    (1, 4, 2, 700, "prefix", 300, 15.0, False),
    (1, 2, 1, 1000, "causal", 1, 0.0, False),
    (4, 40, 20, 300, "causal", 0, 0.0, False),      # more items than SMs
    (5, 40, 40, 140, "docs", 0, 50.0, False),
    (1, 2, 1, 2111, "causal", 0, 30.0, True),
    (1, 3, 1, 1500, "full", 0, 0.0, False),
    (2, 1, 1, 1200, "random", 0, 0.0, True),
    (7, 16, 16, 200, "full", 0, 0.0, False),
    (2, 160, 20, 270, "prefix", 0, 0.0, False),
]


def call(case, d, seed=None):
    B, H, Hkv, N, kind, window, cap, slopes = case
    x = inputs(B, H, Hkv, N, d, cap, 100 + N if seed is None else seed)
    begin, end, causal = masks(kind, B, N, N)
    return x, dict(key_begin=begin, key_end=end, causal=causal, window=window, cap=cap, slopes=slopes_of(H, slopes))


def dev(options):
    return {n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in options.items()}


def plain(options):
    return [options[n] for n in ("key_begin", "key_end", "causal", "window", "cap", "slopes")]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CASES)
def test_forward(case, d):
    x, options = call(case, d)
    q, k, v, _ = (t.cuda() for t in x)
    scale = 1 / math.sqrt(d)
    o, lse = fa.span_attention_forward(q, k, v, scale, **dev(options))
    check_fwd(q, k, v, o, lse, scale, *plain(options))
    again = fa.span_attention_forward(q, k, v, scale, **dev(options))
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CASES)
def test_backward(case, d):
    x, options = call(case, d)
    q, k, v, do = (t.cuda() for t in x)
    scale = 1 / math.sqrt(d)
    o, lse = fa.span_attention_forward(q, k, v, scale, **dev(options))
    grads = fa.span_attention_backward(q, k, v, o, do, lse, scale, **dev(options))
    check_bwd(q, k, v, o, do, lse, grads, scale, *plain(options))
    again = fa.span_attention_backward(q, k, v, o, do, lse, scale, **dev(options))
    assert torch.equal(grads[1], again[1]) and torch.equal(grads[2], again[2])


@pytest.mark.parametrize("d", [64, 128])
def test_backward_against_differences(d):
    """sum(grad u) against the oracle forward's difference along u."""
    case = (1, 2, 1, 150, "docs", 40, 5.0, True)
    (q, k, v, do), options = call(case, d, 50)
    scale = 1 / math.sqrt(d)
    x = [t.cuda() for t in (q, k, v, do)]
    o, lse = fa.span_attention_forward(*x[:3], scale, **dev(options))
    grads = fa.span_attention_backward(*x[:3], o, x[3], lse, scale, **dev(options))
    seen = seen_of(options["key_begin"], options["key_end"], True, 40, 0, 150)
    x0 = [host(t) for t in (q, k, v)]

    def f(x):
        return sum((span_attention_ref(x[0][0, h], x[1][0, 0], x[2][0, 0], scale, seen, 5.0,
                                       float(options["slopes"][h]))[0] * host(do[0, h])).sum() for h in range(2))

    for i, name in enumerate(("dq", "dk", "dv")):
        u = np.random.default_rng(i).standard_normal(x0[i].shape)
        up, down = list(x0), list(x0)
        up[i], down[i] = x0[i] + 1e-4 * u, x0[i] - 1e-4 * u
        diff = (f(up) - f(down)) / 2e-4
        g = host(grads[i])
        # each entry within a few half steps of its size (O enters through delta rounded to bf16): a direction's
        # sum is random over the entries
        assert abs((g * u).sum() - diff) <= 16 * H2 * np.linalg.norm(g), (name, (g * u).sum(), diff)


def test_large_scores_meet_the_cap():
    """Scores far beyond the cap, of both signs, where the tanh is 1 to the last bit."""
    q, k, v, do = (x.cuda() for x in inputs(1, 2, 1, 200, 128, 0.0, 5))
    q, k = (q.float() * 40).bfloat16(), (k.float() * 40).bfloat16()
    o, lse = fa.span_attention_forward(q, k, v, 1.0, causal=True, cap=8.0)
    check_fwd(q, k, v, o, lse, 1.0, None, None, True, 0, 8.0, None)
    grads = fa.span_attention_backward(q, k, v, o, do, lse, 1.0, causal=True, cap=8.0)
    for g in grads[:2]:
        assert torch.isfinite(g).all()
    check_bwd(q, k, v, o, do, lse, grads, 1.0, None, None, True, 0, 8.0, None)


def test_scores_around_the_cap():
    """Scores from far below to twice the cap in the same rows."""
    q, k, v, do = (x.cuda() for x in inputs(2, 4, 2, 300, 64, 0.0, 6))
    k = (k.float() * torch.logspace(-3, 0.7, 300, device="cuda")[None, None, :, None]).bfloat16()
    for cap in (0.5, 2.0, 7.0):
        o, lse = fa.span_attention_forward(q, k, v, 0.3, cap=cap)
        check_fwd(q, k, v, o, lse, 0.3, None, None, False, 0, cap, None)
        grads = fa.span_attention_backward(q, k, v, o, do, lse, 0.3, cap=cap)
        check_bwd(q, k, v, o, do, lse, grads, 0.3, None, None, False, 0, cap, None)


def test_bias_of_far_keys():
    """A slope of 1 over 5000 tokens, a growing bias (negative slope) and none, as three heads."""
    N = 5000
    q, k, v, _ = (x.cuda() for x in inputs(1, 3, 3, N, 64, 0.0, 8))
    slopes = torch.tensor([1.0, -0.01, 0.0])
    o, lse = fa.span_attention_forward(q, k, v, 0.125, causal=True, slopes=slopes.cuda())
    check_fwd(q, k, v, o, lse, 0.125, None, None, True, 0, 0.0, slopes)


def test_keys_outside_all_spans_hold_anything():
    """Padding behind the documents and in front of them, of whole blocks and of parts."""
    B, H, Hkv, N, d = 2, 4, 2, 600, 128
    q, k, v, _ = (x.cuda() for x in inputs(B, H, Hkv, N, d, 0.0, 9))
    begin = torch.full((B, N), 0, dtype=torch.int32)
    end = torch.zeros((B, N), dtype=torch.int32)
    begin[0, :400], end[0, :400] = 0, 400
    begin[1, 150:], end[1, 150:] = 150, 600
    want = None
    for fill in (0.0, float("nan"), float("inf"), torch.finfo(torch.bfloat16).min):
        k[0, :, 400:], v[0, :, 400:], k[1, :, :150], v[1, :, :150] = fill, fill, fill, fill
        o, lse = fa.span_attention_forward(q, k, v, 0.1, begin.cuda(), end.cuda(), causal=True)
        want = want or (o, lse)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), fill
        assert (o[0, :, 400:] == 0).all() and torch.isneginf(lse[1, :, :150]).all()


def test_hidden_scores_may_be_anything():
    """Infinite and NaN scores of pairs outside the spans, in blocks that have others."""
    q, k, v, _ = (x.cuda() for x in inputs(1, 2, 2, 300, 64, 0.0, 12))
    ref = fa.span_attention_forward(q, k, v, 0.125, causal=True)
    k2 = k.clone()
    k2[:, :, 250:] = float("nan")
    k2[:, :, 200:250] = float("inf")
    got = fa.span_attention_forward(q, k2, v, 0.125, causal=True)
    assert torch.equal(got[0][:, :, :200], ref[0][:, :, :200]) and torch.equal(got[1][:, :, :200], ref[1][:, :, :200])


def test_empty_spans_have_no_gradient():
    q, k, v, do = (x.cuda() for x in inputs(1, 4, 2, 200, 64, 0.0, 10))
    begin = torch.full((1, 200), 200, dtype=torch.int32, device="cuda")
    o, lse = fa.span_attention_forward(q, k, v, 0.1, begin)
    assert (o == 0).all() and torch.isneginf(lse).all()
    for g in fa.span_attention_backward(q, k, v, o, do, lse, 0.1, begin):
        assert (g == 0).all()


def test_the_square_forward_is_a_span():
    """Causal spans of one document against fa_fwd: the same rounding bounds on both sides."""
    q, k, v, do = (x.cuda() for x in inputs(2, 3, 3, 900, 128, 0.0, 11))
    a, b = fa.attention_forward(q, k, v, 0.09, causal=True), fa.span_attention_forward(q, k, v, 0.09, causal=True)
    assert (a[0].float() - b[0].float()).abs().max() <= 4 * H2 * v.float().abs().max()
    assert (a[1] - b[1]).abs().max() <= 1e-4


def test_replayed_graph_and_other_stream():
    """Captured steps, replayed with other spans and inputs; two graphs share a workspace."""
    B, H, Hkv, N, d = 2, 4, 2, 400, 128
    q, k, v, do = (x.cuda() for x in inputs(B, H, Hkv, N, d, 0.0, 77))
    begin, end, causal = masks("docs", B, N, 1)
    b, e = begin.cuda(), end.cuda()
    o, lse = torch.empty_like(q), torch.empty((B, H, N), device="cuda")
    g = [torch.empty_like(x) for x in (q, k, v)]
    n = max(fa.fa_span_fwd_workspace_bytes(B, H, Hkv, N, d), fa.fa_span_bwd_workspace_bytes(B, H, Hkv, N, d))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def forward(stream=None):
        fa.fa_span_fwd(q, k, v, b, e, o, lse, ws, 0.1, causal=True, stream=stream)

    def backward(stream=None):
        fa.fa_span_bwd(q, k, v, b, e, o, do, lse, *g, ws, 0.1, causal=True, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    forward(side), backward(side)
    torch.cuda.synchronize()
    check_bwd(q, k, v, o, do, lse, g, 0.1, begin, end, True, 0, 0.0, None)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, step in zip(graphs, (forward, backward)):
        with torch.cuda.graph(graph):
            step()
    for seed in (2, 3):
        begin, end, _ = masks("docs", B, N, seed)
        b.copy_(begin), e.copy_(end), q.copy_(torch.randn_like(q))
        for _ in range(2):
            graphs[0].replay(), graphs[1].replay()
        torch.cuda.synchronize()
        assert fa.fa_check_device_status() == fa.FA_OK
        check_fwd(q, k, v, o, lse, 0.1, begin, end, True, 0, 0.0, None)
        check_bwd(q, k, v, o, do, lse, g, 0.1, begin, end, True, 0, 0.0, None)


@pytest.mark.parametrize("case", [(1, 1, 1, 1), (1, 2, 1, 129), (2, 8, 2, 300), (1, 4, 1, 1500), (3, 40, 20, 140)])
def test_calls_stay_within_their_workspaces(case):
    B, H, Hkv, N = case
    q, k, v, do = (x.cuda() for x in inputs(B, H, Hkv, N, 64, 0.0, 13))
    begin, end, _ = masks("random", B, N, N)
    for backward in (False, True):
        size = (fa.fa_span_bwd_workspace_bytes if backward else fa.fa_span_fwd_workspace_bytes)(B, H, Hkv, N, 64)
        memory = torch.full((size + (1 << 20),), 90, dtype=torch.uint8, device="cuda")
        args = dict(key_begin=begin.cuda(), key_end=end.cuda(), workspace=memory[:size])
        if backward:
            grads = fa.span_attention_backward(q, k, v, o, do, lse, 0.125, **args)
            check_bwd(q, k, v, o, do, lse, grads, 0.125, begin, end, False, 0, 0.0, None)
        else:
            o, lse = fa.span_attention_forward(q, k, v, 0.125, **args)
            check_fwd(q, k, v, o, lse, 0.125, begin, end, False, 0, 0.0, None)
        assert (memory[size:] == 90).all()


def test_two_calls_at_once():
    """Calls on two streams with workspaces of their own."""
    q, k, v, do = (x.cuda() for x in inputs(2, 8, 2, 700, 128, 0.0, 14))
    begin, end, _ = masks("docs", 2, 700, 3)
    args = dict(key_begin=begin.cuda(), key_end=end.cuda(), causal=True, check_status=False)
    want = fa.span_attention_forward(q, k, v, 0.1, **args)
    wantg = fa.span_attention_backward(q, k, v, want[0], do, want[1], 0.1, **args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):
        for s in streams:
            outs.append((fa.span_attention_forward(q, k, v, 0.1, stream=s, **args),
                         fa.span_attention_backward(q, k, v, want[0], do, want[1], 0.1, stream=s, **args)))
    torch.cuda.synchronize()
    assert fa.fa_check_device_status() == fa.FA_OK
    for (o, lse), g in outs:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(g[1], wantg[1]) and torch.equal(g[2], wantg[2])


@pytest.mark.parametrize("N, cap", [(100, 0.0), (700, 0.0), (700, 50.0)])
@pytest.mark.parametrize("window", [0, 2 ** 31 - 1])
def test_spans_of_any_integers(N, cap, window):
    """Values outside [0, N], up to those of the type, give the bits of 0 and N."""
    B, H, Hkv, d = 2, 4, 2, 64
    g = np.random.default_rng(N)
    some = np.array([-2 ** 31, -2 ** 31 + 1, -2 ** 30, -1, 0, 1, N // 2, N, N + 1, 2 ** 30, 2 ** 31 - 1], np.int64)
    begin, end = (torch.from_numpy(g.choice(some, (B, N)).astype(np.int32)).cuda() for _ in range(2))
    begin[0], end[1] = -2 ** 31, 2 ** 31 - 1
    q, k, v, do = (randn(i, B, h, N, d).cuda() for i, h in enumerate((H, Hkv, Hkv, H)))
    outs = []
    for b, e in ((begin, end), (begin.clamp(0, N), end.clamp(0, N))):
        o, lse = fa.span_attention_forward(q, k, v, 0.125, b, e, window=window, cap=cap)
        outs.append((o, lse, *fa.span_attention_backward(q, k, v, o, do, lse, 0.125, b, e, window=window, cap=cap)))
    seen = (begin.clamp(0, N) < end.clamp(0, N))[:, None].expand(B, H, N)
    o, lse, dq, dk, dv = outs[0]
    assert (o[~seen] == 0).all() and (lse[~seen] == -math.inf).all() and (dq[~seen] == 0).all()
    for x, y in zip((o, lse, dk, dv), (outs[1][0], outs[1][1], outs[1][3], outs[1][4])):
        assert torch.equal(x, y)
    # (dQ is summed in any order, in 32 bits, and rounded to bf16)
    torch.testing.assert_close(dq.float(), outs[1][2].float(), rtol=2 ** -7, atol=1e-5 * float(dq.float().abs().max()))
