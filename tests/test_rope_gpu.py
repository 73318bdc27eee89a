"""Head norm and rotation (fa_rope_fwd, fa_rope_bwd) against the fp64 oracle.

Bounds, elementwise, with H = 2^-8 (bf16's half step): one rounding of a value y
is off by H |y|.  fp32 inside: cos and sin to 2^-22 and about ten roundings of
2^-24 of values no larger than the pair's, so 2^-20 of the row's largest value
covers them.  Weight gradients are fp32 sums of n products in a tree of at most
n / 600 + 700 additions a partial: (n / 600 + 700) 2^-24 of the sum of sizes.
"""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from exact_tiled_attention_08_gb300 import fa
from oracle.cross import rope_bwd_ref, rope_ref

pytestmark = pytest.mark.gpu

H2 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_tiled_attention_08_gb300.build import build_library

    build_library()
    fa.load_library()
    assert torch.cuda.is_available()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def close(got, ref, what):
    err = np.abs(got - ref)
    bound = H2 * np.abs(ref) + 2.0 ** -20 * np.abs(ref).max(-1, keepdims=True) + 1e-30
    assert (err <= bound).all(), (what, (err - bound).max())


CASES = [
    # B, N, H, Hkv, d, rot, eps, interleaved, far
    (1, 1, 1, 1, 64, 64, None, False, 0),
    (2, 7, 4, 2, 128, 128, 1e-6, False, 5),
    (1, 33, 3, 1, 128, 64, 1e-5, True, 1000000),
    (3, 5, 2, 2, 64, 16, None, True, 2147483000),
    (2, 130, 5, 1, 128, 96, 1e-6, False, 100000),
    (1, 9, 2, 1, 64, 48, 1e-6, False, 3),
    (2, 17, 8, 2, 128, 0, 1e-6, False, 0),
    (1, 2000, 8, 2, 128, 32, None, False, 77),
    (1, 9001, 11, 3, 64, 64, 1e-6, True, 10),   # units of several heads
    (2, 6000, 3, 20, 128, 128, 1e-6, False, 0),
]


def setup(case, seed=0):
    B, N, H, Hkv, d, rot, eps, inter, far = case
    rows = randn(seed, B, N, H + 2 * Hkv, d)
    q, k, v = rows[:, :, :H], rows[:, :, H:H + Hkv], rows[:, :, H + Hkv:]
    g = torch.Generator().manual_seed(seed + 1)
    w = [None, None] if eps is None else [torch.rand(d, generator=g).cuda() + 0.5 for _ in range(2)]
    freq = fa.rope_frequencies(rot)[0] if rot else None
    pos = (torch.randint(0, far + 1, (B, 1), generator=g) + torch.arange(N)).to(torch.int32).cuda()
    return q, k, v, w, freq, pos


def oracle_args(case, w, freq, pos, b, factor):
    _, _, _, _, _, rot, eps, inter, _ = case
    return (None if w is None else w.cpu().numpy(), freq.cpu().numpy() if rot else np.zeros(0), pos[b].cpu().numpy(),
            eps, factor, inter)


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    B, N, H, Hkv, d, rot, eps, inter, far = case
    q, k, v, w, freq, pos = setup(case)
    C = N + 11
    starts = torch.randint(0, 12, (B,), generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    qo = torch.empty((B, H, N, d), dtype=torch.bfloat16, device="cuda")
    ko = torch.full((B, Hkv, C, d), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full_like(ko, 7.0)
    fa.fa_rope_fwd(q, k, v, *w, freq, pos, starts, qo, ko, vo, eps=eps, factor=1.25, interleaved=inter)
    for b in range(B):
        s = int(starts[b])
        new = slice(s, s + N)
        rest = [r for r in range(C) if not s <= r < s + N]
        close(host(qo[b]), rope_ref(host(q[b].transpose(0, 1)), *oracle_args(case, w[0], freq, pos, b, 1.25)), "q")
        close(host(ko[b, :, new]), rope_ref(host(k[b].transpose(0, 1)), *oracle_args(case, w[1], freq, pos, b, 1.25)), "k")
        assert torch.equal(vo[b, :, new], v[b].transpose(0, 1))
        assert (ko[b][:, rest] == 7).all() and (vo[b][:, rest] == 7).all()


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    B, N, H, Hkv, d, rot, eps, inter, far = case
    q, k, v, w, freq, pos = setup(case)
    gq, gk, gv = randn(5, B, H, N, d), randn(6, B, Hkv, N, d), randn(7, B, Hkv, N, d)
    drows = torch.full((B, N, H + 2 * Hkv + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    dq, dk, dv = drows[:, :, :H], drows[:, :, H:H + Hkv], drows[:, :, H + Hkv:-1]
    dw = [None, None] if eps is None else [torch.empty(d, device="cuda") for _ in range(2)]
    ws = torch.full((fa.fa_rope_bwd_workspace_bytes(B, H, Hkv, N, d),), 255, dtype=torch.uint8, device="cuda")
    call = lambda: fa.fa_rope_bwd(q, k, *w, freq, pos, gq, gk, gv, dq, dk, dv, *dw, ws, eps=eps, factor=1.25,
                                  interleaved=inter)
    call()
    for x, wt, g, dx, dwt, name in ((q, w[0], gq, dq, dw[0], "q"), (k, w[1], gk, dk, dw[1], "k")):
        total, size = np.zeros(d), np.zeros(d)
        for b in range(B):
            args = oracle_args(case, wt, freq, pos, b, 1.25)
            xb, gb = host(x[b].transpose(0, 1)), host(g[b])
            ref, rw = rope_bwd_ref(xb, args[0], args[1], args[2], gb, *args[3:])
            got = host(dx[b].transpose(0, 1))
            err = np.abs(got - ref)
            # the norm's gradient subtracts the row's projection: sizes of both terms, not of their difference
            bound = H2 * np.abs(ref) + 2.0 ** -19 * (np.abs(ref).max(-1, keepdims=True) + np.abs(gb).max(-1, keepdims=True) * 4)
            assert (err <= bound).all(), (name, (err - bound).max())
            if eps is not None:
                total += rw
                inv = 1 / np.sqrt((xb * xb).mean(-1, keepdims=True) + eps)
                size += (np.linalg.norm(gb, axis=-1, keepdims=True) * 1.25 * np.abs(xb * inv)).reshape(-1, d).sum(0)
        if eps is not None:
            n = B * N * x.shape[2]
            err = np.abs(host(dwt) - total)
            assert (err <= (n / 600 + 700) * 2.0 ** -24 * size).all(), (name, (err / size).max())
    assert torch.equal(dv, gv.transpose(1, 2)) and (drows[:, :, -1] == 7).all()
    first = [t.clone() for t in (drows, *dw) if t is not None]
    call()
    assert all(torch.equal(a, b) for a, b in zip(first, (t for t in (drows, *dw) if t is not None)))


def test_backward_against_differences():
    case = (1, 6, 2, 1, 64, 32, 1e-3, True, 50)
    B, N, H, Hkv, d, rot, eps, inter, far = case
    q, k, v, w, freq, pos = setup(case)
    gq = randn(5, B, H, N, d)
    dq, dw = torch.empty((B, N, H, d), dtype=torch.bfloat16, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(fa.fa_rope_bwd_workspace_bytes(B, H, Hkv, N, d), dtype=torch.uint8, device="cuda")
    fa.fa_rope_bwd(q, None, w[0], None, freq, pos, gq, None, None, dq, None, None, dw, None, ws, eps=eps,
                   interleaved=inter)
    x, wt, g = host(q[0].transpose(0, 1)), w[0].cpu().numpy().astype(np.float64), host(gq[0])

    def f(x, wt):
        return (rope_ref(x, wt, freq.cpu().numpy(), pos[0].cpu().numpy(), eps, 1.0, inter) * g).sum()

    rng, h = np.random.default_rng(0), 1e-5
    u, uw = rng.standard_normal(x.shape), rng.standard_normal(d)
    got = host(dq[0].transpose(0, 1))
    diff = (f(x + h * u, wt) - f(x - h * u, wt)) / (2 * h)
    assert abs((got * u).sum() - diff) <= H2 * np.abs(got * u).sum()  # each entry off by half a step
    diff = (f(x, wt + h * uw) - f(x, wt - h * uw)) / (2 * h)
    assert abs((host(dw) * uw).sum() - diff) <= 1e-5 * np.abs(host(dw) * uw).sum() + 1e-4


def test_parts_left_out_and_rows_past_the_capacity():
    case = (2, 4, 2, 1, 64, 64, None, False, 0)
    q, k, v, w, freq, pos = setup(case)
    qo = torch.empty((2, 2, 4, 64), dtype=torch.bfloat16, device="cuda")
    fa.fa_rope_fwd(q, None, None, None, None, freq, pos, None, qo, None, None)
    close(host(qo[1]), rope_ref(host(q[1].transpose(0, 1)), None, freq.cpu().numpy(), pos[1].cpu().numpy()), "q")
    ko, vo = torch.full((2, 1, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((2, 1, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    starts = torch.tensor([2, -3], dtype=torch.int32, device="cuda")
    fa.fa_rope_fwd(None, k, v, None, None, None, None, starts, None, ko, vo)  # no rotation, no norm: moved
    assert torch.equal(ko[0, :, 2:], k[0, :2].transpose(0, 1)) and (ko[0, :, :2] == 7).all()
    assert torch.equal(vo[1, :, 0], v[1, 3]) and (vo[1, :, 1:] == 7).all()
    # without positions a token's place in the cache is its position
    fa.fa_rope_fwd(None, k, v, None, None, freq, None, starts, None, ko, vo)
    close(host(ko[0, :, 2:]), rope_ref(host(k[0, :2].transpose(0, 1)), None, freq.cpu().numpy(), [2, 3]), "k")


def test_broadcast_inputs_and_zero_rows():
    """Keys of one head broadcast over the tokens (stride 0); a row of zeros under the norm."""
    freq = fa.rope_frequencies(64)[0]
    one = randn(1, 1, 1, 2, 64)
    k = one.expand(2, 5, 2, 64)
    ko = torch.empty((2, 2, 5, 64), dtype=torch.bfloat16, device="cuda")
    fa.fa_rope_fwd(None, k, None, None, None, freq, None, None, None, ko, None)
    close(host(ko[1]), rope_ref(host(k[1].transpose(0, 1)), None, freq.cpu().numpy(), np.arange(5)), "k")
    z = torch.zeros((1, 3, 1, 64), dtype=torch.bfloat16, device="cuda")
    qo = torch.empty((1, 1, 3, 64), dtype=torch.bfloat16, device="cuda")
    fa.fa_rope_fwd(z, None, None, None, None, freq, None, None, qo, None, None, eps=1e-6)
    assert (qo == 0).all()


@pytest.mark.parametrize("scaling", [None, "linear", "base", "parts"])
def test_scaled_frequencies(scaling):
    freq, factor = fa.rope_frequencies(128, 10000.0, scaling=scaling, scale=8.0 if scaling else 1.0, trained_len=4096,
                                       device="cpu")
    plain = 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)
    if scaling is None:
        assert torch.equal(freq, plain)
    elif scaling == "linear":
        assert torch.allclose(freq * 8, plain, rtol=1e-14)
    else:
        assert math.isclose(float(freq[0]), 1.0) and math.isclose(float(freq[-1] * 8), float(plain[-1]), rel_tol=1e-12)
    assert factor == (0.1 * math.log(8) + 1 if scaling == "parts" else 1.0)


def test_replayed_graph():
    case = (2, 40, 4, 2, 128, 128, 1e-6, False, 9)
    B, N, H, Hkv, d, *_ = case
    q, k, v, w, freq, pos = setup(case)
    outs = [torch.empty((B, h, N, d), dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv)]
    call = lambda: fa.fa_rope_fwd(q, k, v, *w, freq, pos, None, *outs, eps=1e-6)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    pos.add_(1000)
    graph.replay()
    for b in range(B):
        close(host(outs[0][b]), rope_ref(host(q[b].transpose(0, 1)), *oracle_args(case, w[0], freq, pos, b, 1.0)), "q")


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("position", [0, 1, 4097, 2 ** 24 + 1, 2 ** 31 - 1, -1, -2 ** 31])
def test_angles_at_far_positions(position, interleaved):
    """cos and sin as the gradient of a weight sees them, in fp32: a row of ones, of
    which the first of each pair has a gradient of 1, gives cos and -sin.
    Bound: the angle's 2^-23 + 2^-52 |position freq|, and 2^-21 for sincospi (1 ulp), the norm's
    reciprocal root (2 ulp) and four roundings."""
    d = 128
    freq, _ = fa.rope_frequencies(d)
    q = torch.ones((1, 1, 1, d), dtype=torch.bfloat16, device="cuda")
    first = torch.arange(d, device="cuda") % 2 == 0 if interleaved else torch.arange(d, device="cuda") < d // 2
    dy = first.bfloat16().reshape(1, 1, 1, d).contiguous()
    dq, dw = torch.empty_like(q), torch.empty((d,), device="cuda")
    ws = torch.empty(fa.fa_rope_bwd_workspace_bytes(1, 1, 1, 1, d), dtype=torch.uint8, device="cuda")
    pos = torch.tensor([[position]], dtype=torch.int32, device="cuda")
    fa.fa_rope_bwd(q, None, None, None, freq, pos, dy, None, None, dq, None, None, dw, None, ws, eps=0.0,
                   interleaved=interleaved)
    got = dw.double().cpu()
    a, b = (got[0::2], got[1::2]) if interleaved else (got[:d // 2], got[d // 2:])
    for i, f in enumerate(freq.tolist()):
        angle = float(2 * PI * (Fraction(f) * position / (2 * PI) % 1))
        bound = 2.0 ** -23 + 2.0 ** -52 * abs(position) * f + 2.0 ** -21
        assert abs(a[i] - math.cos(angle)) <= bound and abs(b[i] + math.sin(angle)) <= bound, (i, f)
