"""Cross attention (fa_cross_fwd, fa_cross_bwd) and attention over a cache
(fa_tree_fwd) against the fp64 oracle.

Bounds, elementwise.  H = 2^-8 is the half step of bf16.
  O    each P is rounded to bf16 before it meets V and O once at the end, and the
       normaliser differs from the sum of the rounded P by at most H of it:
       H (A + 2 |O|) with A = sum_j P_j |v_j|; fp32 scores, exponentials and
       sums add at most 1e-4 A (scores below 2^4 in magnitude: (d + 2) 2^-24
       times sum |q k| scale < 2^3 gives 6e-5, twice 2^-22 each for the
       exponential and its argument).
  LSE  1e-4 by the same, plus fp32's 2^-22 |LSE|.
  dV   H (sum_i P |dO| + |dV|) + 2e-4 sum P |dO|
  dQ   H (scale sum_j |dS| |k| + |dQ|) + 2e-4 scale sum_j P (|dO| |v| + |dO o|) |k|
       for the rounding of dS and of dQ and the fp32 error of P and dP - delta;
  dK   the same with q.  Sums over a group's heads add up.
"""

import math

import numpy as np
import pytest
import torch

from exact_tiled_attention_08_gb300 import fa
from oracle.cross import masked_attention_bwd_ref, masked_attention_ref, tree_visible

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


def cross_inputs(B, H, Hkv, Nq, Nk, d, seed):
    return randn(seed, B, H, Nq, d), randn(seed + 1, B, Hkv, Nk, d), randn(seed + 2, B, Hkv, Nk, d), \
        randn(seed + 3, B, H, Nq, d)


def heads_of(B, H):
    """(b, h) pairs to check: all of them, or a spread of twelve."""
    every = [(b, h) for b in range(B) for h in range(H)]
    return every if len(every) <= 12 else [every[i * (len(every) - 1) // 11] for i in range(12)]


def check_rows(o, lse, ref, what):
    ro, rl, size = ref
    err = np.abs(o - ro)
    bound = H2 * (size + 2 * np.abs(ro)) + 1e-4 * size
    assert (err <= bound).all(), (what, "o", (err - bound).max())
    dead = np.isneginf(rl)
    assert np.isneginf(lse[dead]).all() and (o[dead] == 0).all(), what
    err = np.abs(lse[~dead] - rl[~dead])
    assert (err <= 1e-4 + 2.0 ** -22 * np.abs(rl[~dead])).all(), (what, "lse", err.max())


def check_cross_fwd(q, k, v, o, lse, scale, lens):
    B, H, Nq, _ = q.shape
    G, Nk = H // k.shape[1], k.shape[2]
    for b, h in heads_of(B, H):
        seen = np.zeros((Nq, Nk), bool)
        seen[:, :Nk if lens is None else lens[b]] = True
        ref = masked_attention_ref(host(q[b, h]), host(k[b, h // G]), host(v[b, h // G]), scale, seen)
        check_rows(host(o[b, h]), host(lse[b, h]), ref, (b, h))


CROSS = [
    # B, H, Hkv, Nq, Nk, lens
    (1, 1, 1, 1, 1, None),
    (1, 2, 1, 1, 77, None),
    (2, 4, 2, 3, 129, [129, 1]),
    (3, 2, 2, 127, 128, [0, 64, 128]),
    (2, 6, 2, 50, 300, [300, 128]),
    (1, 4, 4, 129, 257, None),
    (1, 8, 2, 64, 200, None),        # 256 rows share a key/value head
    (2, 5, 1, 103, 513, [513, 400]),  # 515 rows
    (4, 2, 1, 1, 5000, [5000, 3, 0, 2600]),
    (1, 1, 1, 1, 40000, None),
    (1, 1, 1, 700, 6000, None),      # few rows of blocks, many keys
    (5, 16, 8, 40, 260, [1, 255, 256, 257, 260]),
    (2, 40, 40, 130, 384, [384, 130]),  # more items than SMs
    (4, 40, 40, 2, 1500, [1500, 700, 1499, 64]),  # many key blocks a CTA
    (2, 40, 20, 130, 1111, None),
    # few items with equal lengths: CTAs of a cluster share an item
    (1, 8, 8, 1, 1500, None),
    (4, 16, 16, 2, 129, None),
    (1, 40, 20, 60, 2000, None),
    (2, 16, 8, 16, 700, None),
    (1, 3, 1, 40, 900, [899]),
    (1, 72, 72, 128, 1300, None),
    (1, 2, 2, 5, 300, [0]),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CROSS)
def test_cross_forward(case, d):
    B, H, Hkv, Nq, Nk, lens = case
    q, k, v, _ = (x.cuda() for x in cross_inputs(B, H, Hkv, Nq, Nk, d, 100 + Nq + Nk))
    scale = 1 / math.sqrt(d)
    kl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.cross_attention_forward(q, k, v, scale, kl)
    check_cross_fwd(q, k, v, o, lse, scale, lens)
    again = fa.cross_attention_forward(q, k, v, scale, kl)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def check_cross_bwd(q, k, v, o, do, lse, grads, scale, lens):
    B, H, Nq, _ = q.shape
    Hkv, Nk = k.shape[1:3]
    G = H // Hkv
    dq, dk, dv = grads
    for b, j in heads_of(B, Hkv):
        n = Nk if lens is None else lens[b]
        seen = np.zeros((Nq, Nk), bool)
        seen[:, :n] = True
        sums = [np.zeros((3, Nk, q.shape[3])) for _ in range(2)]
        for h in range(j * G, (j + 1) * G):
            g, half, fp32 = masked_attention_bwd_ref(*(host(x) for x in (q[b, h], k[b, j], v[b, j], o[b, h], do[b, h],
                                                                         lse[b, h])), scale, seen)
            err = np.abs(host(dq[b, h]) - g[0])
            bound = H2 * (half[0] + np.abs(g[0])) + 2e-4 * fp32[0] + 1e-30
            assert (err <= bound).all(), (b, h, "dq", (err - bound).max(), err.max())
            for i in (0, 1):
                sums[i] += np.stack([g[1 + i], half[1 + i], fp32[1 + i]])
        for name, got, (g, half, fp32) in (("dk", dk, sums[0]), ("dv", dv, sums[1])):
            got = host(got[b, j])
            assert (got[n:] == 0).all(), (b, j, name)
            err = np.abs(got - g)
            bound = H2 * (half + np.abs(g)) + 2e-4 * fp32 + 1e-30
            assert (err <= bound).all(), (b, j, name, (err - bound).max(), err.max())


CROSS_BWD = [c for c in CROSS if c[3] * c[4] < 1000000] + [
    (1, 1, 1, 3000, 40, None),           # one key block: dQ written directly, runs of query blocks
    (3, 4, 2, 300, 128, [128, 0, 5]),
    (2, 2, 2, 77, 100, [0, 0]),
    (1, 2, 1, 900, 1100, [1000]),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CROSS_BWD)
def test_cross_backward(case, d):
    B, H, Hkv, Nq, Nk, lens = case
    q, k, v, do = (x.cuda() for x in cross_inputs(B, H, Hkv, Nq, Nk, d, 300 + Nq + Nk))
    scale = 1 / math.sqrt(d)
    kl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.cross_attention_forward(q, k, v, scale, kl)
    grads = fa.cross_attention_backward(q, k, v, o, do, lse, scale, kl)
    check_cross_bwd(q, k, v, o, do, lse, grads, scale, lens)
    again = fa.cross_attention_backward(q, k, v, o, do, lse, scale, kl)
    assert torch.equal(grads[1], again[1]) and torch.equal(grads[2], again[2])


@pytest.mark.parametrize("d", [64, 128])
def test_cross_backward_against_differences(d):
    """sum(grad u) against the oracle forward's difference along u; the forward is
    exact in fp64, so the gradients' own bounds are what separates them."""
    B, H, Hkv, Nq, Nk, n = 1, 2, 1, 33, 150, 140
    q, k, v, do = cross_inputs(B, H, Hkv, Nq, Nk, d, 50)
    scale = 1 / math.sqrt(d)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    dev = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.cross_attention_forward(*dev[:3], scale, lens)
    grads = fa.cross_attention_backward(*dev[:3], o, dev[3], lse, scale, lens)
    seen = np.zeros((Nq, Nk), bool)
    seen[:, :n] = True
    x0 = [host(t) for t in (q, k, v)]

    def f(x):
        return sum((masked_attention_ref(x[0][0, h], x[1][0, 0], x[2][0, 0], scale, seen)[0] * host(do[0, h])).sum()
                   for h in range(H))

    for i, name in enumerate(("dq", "dk", "dv")):
        u = np.random.default_rng(i).standard_normal(x0[i].shape)
        step = 1e-4
        up, down = [list(x0), list(x0)]
        up[i] = x0[i] + step * u
        down[i] = x0[i] - step * u
        diff = (f(up) - f(down)) / (2 * step)
        g = host(grads[i])
        # O enters through delta rounded to bf16: H |dO| . |O| per row more than the kernel's own bounds,
        # all below 4 H of the norms; a direction's sum is random over the entries
        assert abs((g * u).sum() - diff) <= 4 * H2 * np.linalg.norm(g) * 4, (name, (g * u).sum(), diff)


@pytest.mark.parametrize("d", [64, 128])
def test_padding_holds_anything(d):
    """NaN and infinities behind the keys change nothing, forward and backward."""
    B, H, Hkv, Nq, Nk, lens = 3, 4, 2, 70, 400, [0, 130, 257]
    q, k, v, do = (x.cuda() for x in cross_inputs(B, H, Hkv, Nq, Nk, d, 9))
    kl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = None
    for fill in (0.0, float("nan"), float("inf"), torch.finfo(torch.bfloat16).min):
        for b, n in enumerate(lens):
            k[b, :, n:] = fill
            v[b, :, n:] = fill
        o, lse = fa.cross_attention_forward(q, k, v, 0.1, kl)
        dq, dk, dv = fa.cross_attention_backward(q, k, v, o, do, lse, 0.1, kl)
        if want is None:
            want = o, lse, dk, dv, dq
        for got, ref in zip((o, lse, dk, dv), want):
            assert torch.equal(got, ref), fill
        # (dQ sums its blocks' parts in any order: each within fp32's rounding, then one bf16 step)
        assert torch.allclose(dq.float(), want[4].float(), rtol=2 * H2, atol=1e-5), fill
        assert (o[0] == 0).all() and torch.isneginf(lse[0]).all() and (dq[0] == 0).all()


def test_lengths_outside_the_keys_are_taken_into_them():
    q, k, v, do = (x.cuda() for x in cross_inputs(2, 2, 1, 5, 140, 64, 3))
    a = fa.cross_attention_forward(q, k, v, 0.1, torch.tensor([-7, 2 ** 31 - 1], dtype=torch.int32, device="cuda"))
    b = fa.cross_attention_forward(q, k, v, 0.1, torch.tensor([0, 140], dtype=torch.int32, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_large_scores_and_infinite_scores():
    """Scores far apart (one key takes all), and keys whose score is -inf."""
    q, k, v, _ = cross_inputs(1, 1, 1, 40, 300, 128, 5)
    q, k, v = (q.float().abs() * 6).bfloat16().cuda(), k.cuda(), v.cuda()
    o, lse = fa.cross_attention_forward(q, k, v, 1.0)
    seen = np.ones((40, 300), bool)
    ro, rl, size = masked_attention_ref(host(q[0, 0]), host(k[0, 0]), host(v[0, 0]), 1.0, seen)
    # scores up to 2^11: their fp32 sums are off by 130 2^-24 sum |q k| < 2^-4 in the worst case
    # (all roundings one way); P is off by twice that relatively
    worst = 130 * 2.0 ** -24 * (np.abs(host(q[0, 0])) @ np.abs(host(k[0, 0])).T).max()
    err = np.abs(host(o[0, 0]) - ro)
    assert (err <= H2 * (size + 2 * np.abs(ro)) + 3 * worst * np.abs(host(v)).max()).all(), err.max()
    assert np.abs(host(lse[0, 0]) - rl).max() <= worst + 2.0 ** -21 * np.abs(rl).max()
    k[0, 0, 10:] = -math.inf  # q > 0: these scores are -inf
    q.clamp_(min=0.125)
    o, lse = fa.cross_attention_forward(q, k, v, 0.1)
    ref = fa.cross_attention_forward(q, k[:, :, :10].contiguous(), v[:, :, :10].contiguous(), 0.1)
    assert torch.allclose(o.float(), ref[0].float(), rtol=2 * H2, atol=1e-6)
    assert torch.allclose(lse, ref[1], rtol=1e-6, atol=1e-6)
    k[0, 0] = -math.inf
    o, lse = fa.cross_attention_forward(q, k, v, 0.1)
    assert (o == 0).all() and torch.isneginf(lse).all()


TREE = [
    # B, H, Hkv, T, C, lens, drafts, masked
    (1, 1, 1, 1, 2, [0], None, False),
    (1, 8, 2, 1, 300, [255], None, False),
    (2, 4, 2, 5, 260, [126, 255], [5, 3], True),
    (3, 2, 1, 64, 400, [0, 100, 336], [64, 0, 63], True),
    (2, 8, 8, 17, 700, [640, 3], None, False),
    (1, 8, 1, 40, 1000, [900], [39], True),      # 320 rows
    (2, 3, 1, 200, 500, [250, 299], [200, 150], False),
    (4, 16, 8, 7, 5000, [4990, 2000, 0, 129], [7, 7, 2, 7], True),
    (1, 2, 1, 3, 30000, [29000], None, True),
    (2, 2, 2, 8, 64, [60, 64], None, False),     # drafts that do not fit are not there
    (40, 16, 8, 2, 300, list(range(0, 280, 7)), None, True),
    (1, 32, 8, 1, 2048, [1907], None, False),
    (1, 16, 16, 7, 900, [850], [5], True),
    (1, 8, 4, 64, 300, [200], [64], True),
    (1, 4, 2, 3, 1000, [0], [0], False),
    (20, 16, 8, 3, 4000, [3990 - 7 * i for i in range(20)], None, True),  # many key blocks a CTA
]


def tree_inputs(case, d):
    B, H, Hkv, T, C, lens, drafts, masked = case
    q, k, v = randn(T, B, H, T, d), randn(T + 1, B, Hkv, C, d), randn(T + 2, B, Hkv, C, d)
    masks = None
    if masked:
        g = torch.Generator().manual_seed(T)
        parents = torch.stack([torch.randint(-1, n, (B,), generator=g) if n else torch.full((B,), -1) for n in range(T)], 1)
        masks = fa.tree_masks(parents)
    return q, k, v, masks


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", TREE)
def test_tree_forward(case, d):
    B, H, Hkv, T, C, lens, drafts, masked = case
    q, k, v, masks = tree_inputs(case, d)
    have = [min(T if drafts is None else drafts[b], C - lens[b]) for b in range(B)]
    for b in range(B):
        k[b, :, lens[b] + have[b]:] = float("nan")
        v[b, :, lens[b] + have[b]:] = float("inf")
    scale = 1 / math.sqrt(d)
    dev = [x.cuda() for x in (q, k, v)]
    i32 = dict(dtype=torch.int32, device="cuda")
    o = torch.full_like(dev[0], 7.0)
    lse = torch.full((B, H, T), 7.0, device="cuda")
    ws = torch.full((fa.fa_tree_fwd_workspace_bytes(B, H, Hkv, T, C, d),), 255, dtype=torch.uint8, device="cuda")
    fa.fa_tree_fwd(*dev, torch.tensor(lens, **i32), None if drafts is None else torch.tensor(drafts, **i32),
                   None if masks is None else masks.cuda(), o, lse, ws, scale)
    assert fa.fa_check_device_status() == fa.FA_OK
    for b, h in heads_of(B, H):
        m = None if masks is None else [int(w) & (2 ** 64 - 1) for w in masks[b]]
        seen = tree_visible(lens[b], have[b], T, C, m)
        ref = masked_attention_ref(host(q[b, h]), host(k[b, h // (H // Hkv)]), host(v[b, h // (H // Hkv)]), scale, seen)
        n = have[b]
        check_rows(host(o[b, h])[:n], host(lse[b, h])[:n], [x[:n] for x in ref], (b, h))
    for b in range(B):  # rows of tokens that are not there
        assert (o[b, :, have[b]:] == 7).all() and (lse[b, :, have[b]:] == 7).all()


def test_tree_masks_that_leave_a_row_empty():
    """A token of an empty cache that sees nothing, not even itself."""
    q, k, v = (randn(i, 1, 2, 3, 64).cuda() for i in range(3))
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    masks = torch.tensor([[1, 0, 6]], device="cuda")
    o, lse = fa.tree_attention_forward(q, k, v, lens, 0.2, draft_masks=masks)
    assert (o[:, :, 1] == 0).all() and torch.isneginf(lse[:, :, 1]).all()
    assert torch.isfinite(lse[:, :, 0]).all() and torch.equal(o[:, :, 0], v[:, :, 0])


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements; the last request's rows against the first's."""
    B, Hkv, C, d = 3, 2, 3 * 10 ** 6, 128
    k = torch.zeros((B, Hkv, C, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    n = 300
    kk, vv = randn(1, Hkv, n, d).cuda(), randn(2, Hkv, n, d).cuda()
    q = randn(3, 1, 4, 1, d).cuda().expand(B, 4, 1, d).contiguous()
    k[0, :, :n], v[0, :, :n], k[2, :, :n], v[2, :, :n] = kk, vv, kk, vv
    k[1, :, C - n:], v[1, :, C - n:] = kk, vv
    lens = torch.tensor([n - 1, C - 1, n - 1], dtype=torch.int32, device="cuda")
    o, lse = fa.tree_attention_forward(q, k, v, lens, 0.1)
    assert torch.equal(o[0], o[2]) and torch.equal(lse[0], lse[2])
    # request 1: the same keys behind C - n zero rows, whose weight is exp(0) each and whose values are 0
    rest = lse[0].double()
    want = torch.log(torch.exp(rest) + (C - n))
    assert torch.allclose(lse[1].double(), want, atol=1e-4)


def test_replayed_graph_and_other_stream():
    """Captured calls, replayed with other lengths and inputs, on a side stream."""
    B, H, Hkv, Nq, Nk, d = 2, 4, 2, 20, 700, 128
    q, k, v, do = (x.cuda() for x in cross_inputs(B, H, Hkv, Nq, Nk, d, 77))
    lens = torch.tensor([700, 20], dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((B, H, Nq), device="cuda")
    g = [torch.empty_like(x) for x in (q, k, v)]
    wf = torch.empty(fa.fa_cross_fwd_workspace_bytes(B, H, Hkv, Nq, Nk, d), dtype=torch.uint8, device="cuda")
    wb = torch.empty(fa.fa_cross_bwd_workspace_bytes(B, H, Hkv, Nq, Nk, d), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        fa.fa_cross_fwd(q, k, v, lens, o, lse, wf, 0.1, stream)
        fa.fa_cross_bwd(q, k, v, lens, o, do, lse, *g, wb, 0.1, stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in ([3, 700], [0, 129], [700, 700]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        q.copy_(torch.randn_like(q))
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_check_device_status() == fa.FA_OK
        check_cross_fwd(q, k, v, o, lse, 0.1, n)
        check_cross_bwd(q, k, v, o, do, lse, g, 0.1, n)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", [
    (1, 160, 160, 200, 300, None),      # 160 row tile pairs: a full round, then pairs cut into single tiles
    (1, 160, 160, 100, 500, None),      # the same with one row tile per head
    (2, 130, 130, 300, 260, None),      # 520 pairs, a last round of many
    (2, 20, 10, 1100, 200, [200, 190]),  # equal numbers of blocks of unequal lengths
    (1, 250, 250, 129, 3000, None),     # a last round that is cut
    (1, 153, 153, 256, 128, None),
])
def test_rounds_of_equal_items(case, d):
    """More items than CTAs, all with the same number of key blocks."""
    B, H, Hkv, Nq, Nk, lens = case
    q, k, v, _ = (x.cuda() for x in cross_inputs(B, H, Hkv, Nq, Nk, d, 7))
    scale = 1 / math.sqrt(d)
    kl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.cross_attention_forward(q, k, v, scale, kl)
    # every head against fp32, the oracle's spread of twelve by its bounds
    check_cross_fwd(q, k, v, o, lse, scale, lens)
    G = H // Hkv
    s = torch.matmul(q.float(), k.float().repeat_interleave(G, 1).transpose(-1, -2)) * scale
    if lens is not None:
        s = s.masked_fill(torch.arange(Nk, device="cuda") >= kl[:, None, None, None], -math.inf)
    ref = torch.matmul(torch.softmax(s, -1), v.float().repeat_interleave(G, 1))
    assert (o.float() - ref).abs().max() <= 4 * H2 * v.float().abs().max()
    assert (lse - torch.logsumexp(s, -1)).abs().max() <= 1e-3  # (both sides fp32)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 200])
def test_parts_without_keys_before_low_scores(Nq, d):
    """One head's keys in some forty parts; those of the first nine score -inf, the
    others about e^-110 (2^-159, far below the least exponential in fp32)."""
    Nk, dead = 5000, 1150
    # scores (whole numbers) / 8, exact in fp32: what is left is c log2(e)'s rounding, 2^-24 of 112
    q = torch.ones((1, 1, Nq, d), dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(d)
    k = torch.full((1, 1, Nk, d), -896.0 / d)
    k += torch.arange(d) < torch.randint(0, 17, (1, 1, Nk, 1), generator=g)
    k[:, :, :dead] = -math.inf
    q, k, v = q.cuda(), k.bfloat16().cuda(), randn(1, 1, 1, Nk, d).cuda()
    o, lse = fa.cross_attention_forward(q, k, v, 0.125)
    seen = np.ones((Nq, Nk - dead), bool)
    ref = masked_attention_ref(host(q[0, 0]), host(k[0, 0, dead:]), host(v[0, 0, dead:]), 0.125, seen)
    check_rows(host(o[0, 0]), host(lse[0, 0]), ref, Nq)


@pytest.mark.parametrize("Nk", [300, 700, 9000])
@pytest.mark.parametrize("items", [7, 15, 16, 36, 37, 76, 77])
def test_on_either_side_of_the_cluster_rule(items, Nk):
    """One more item than the device holds clusters, and keys that are too many for clusters."""
    q, k, v, _ = (x.cuda() for x in cross_inputs(1, items, items, 3, Nk, 64, items + Nk))
    o, lse = fa.cross_attention_forward(q, k, v, 0.125)
    check_cross_fwd(q, k, v, o, lse, 0.125, None)


@pytest.mark.parametrize("case", [(1, 1, 1, 129, 1), (1, 2, 1, 65, 129), (1, 1, 1, 3000, 40), (2, 4, 2, 300, 500),
                                  (2, 4, 1, 700, 200)])
def test_backward_stays_within_its_workspace(case):
    """Runs of cut items in a workspace of exactly the bytes asked for."""
    B, H, Hkv, Nq, Nk = case
    q, k, v, do = (x.cuda() for x in cross_inputs(B, H, Hkv, Nq, Nk, 64, 11))
    o, lse = fa.cross_attention_forward(q, k, v, 0.125)
    n = fa.fa_cross_bwd_workspace_bytes(B, H, Hkv, Nq, Nk, 64)
    memory = torch.full((n + (1 << 20),), 90, dtype=torch.uint8, device="cuda")
    grads = fa.cross_attention_backward(q, k, v, o, do, lse, 0.125, workspace=memory[:n])
    check_cross_bwd(q, k, v, o, do, lse, grads, 0.125, None)
    assert (memory[n:] == 90).all()
