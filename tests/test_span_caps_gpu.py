"""Capped scores where a row's products are not spread around zero: rows without any product
above zero, rows whose products all lie many caps below it, hidden keys that are much nearer
than every key a row sees.  Spans and pages, with gradients; bounds as in test_span_gpu."""

import math

import pytest
import torch

from exact_tiled_attention_08_gb300 import fa
from test_paged_gpu import check_paged, pool, tables
from test_span_gpu import check_bwd, check_fwd, inputs, masks, randn, slopes_of

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32)


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_tiled_attention_08_gb300.build import build_library

    build_library()
    fa.load_library()


def direction(d):
    return torch.where(torch.rand(d, generator=torch.Generator().manual_seed(d)) < 0.5, -1.0, 1.0)


def shares(caps):
    """Keys' lengths, the longest 1, and what the queries make up for it."""
    top = float(caps.abs().max())
    return (caps / top if top else torch.ones_like(caps)), top


def directed(B, H, Hkv, N, d, caps, cap):
    """q, k, v, do with scale q.k about caps[j] cap for key j of every query, scale = d^-1/2 (keys
    differ by a twentieth of a unit in each channel)."""
    q, k, v, do = inputs(B, H, Hkv, N, d, 0.0, 31)
    u, (rows, top) = direction(d), shares(caps)
    k = ((u + 0.05 * k.float()) * rows[None, None, :, None]).bfloat16()
    q = (u * (cap * top / math.sqrt(d))).bfloat16().expand(B, H, N, d).contiguous()
    return [x.cuda() for x in (q, k, v, do)]


def both_ways(x, kind, cap, d, slopes=None, spans=None):
    q, k, v, do = x
    B, H, N, _ = q.shape
    begin, end, causal = masks(kind, B, N, 5) if spans is None else (*spans, False)
    args = dict(key_begin=None if begin is None else begin.cuda(), key_end=None if end is None else end.cuda(),
                causal=causal, cap=cap, slopes=None if slopes is None else slopes.cuda())
    scale = 1 / math.sqrt(d)
    o, lse = fa.span_attention_forward(q, k, v, scale, **args)
    check_fwd(q, k, v, o, lse, scale, begin, end, causal, 0, cap, slopes)
    grads = fa.span_attention_backward(q, k, v, o, do, lse, scale, **args)
    for g in grads:
        assert torch.isfinite(g).all()
    check_bwd(q, k, v, o, do, lse, grads, scale, begin, end, causal, 0, cap, slopes)


def over_pages(T, pattern, cap, d):
    B, H, Hkv, size, lens = 2, 4, 2, 32, [700, 385]
    table, count = tables(lens, [T] * B, size, -(-(max(lens) + T) // size), 1)
    u, (shared, top) = direction(d).cuda(), shares(caps_of(pattern, max(lens) + T + size))
    kp, vp = pool(1, count, Hkv, size, d, "tokens"), pool(2, count, Hkv, size, d, "heads")
    away = u + 0.05 * kp.float()
    for b, n in enumerate(lens):
        for i in range(-(-(n + T) // size)):
            page = int(table[b, i])
            kp[page] = (away[page] * shared[i * size:(i + 1) * size, None].cuda()).bfloat16()
    q = (u * (cap * top / math.sqrt(d))).bfloat16().expand(B, H, T, d).contiguous()
    scale = 1 / math.sqrt(d)
    o, lse = fa.paged_attention_forward(q, kp, vp, table.cuda(), torch.tensor(lens, **I32).cuda(), scale, cap=cap)
    check_paged(q, kp, vp, table, o, lse, scale, lens, [T] * B, 0, cap, None)


def caps_of(pattern, N):
    """What scale q.k is of each key, in caps."""
    j = torch.arange(N)
    return {"zero": torch.zeros(N),
            "against": torch.full((N,), -0.3),
            "turning": torch.where(j < N // 3, 0.1, -0.3),  # (keys are taken from the last to the first)
            "low": torch.full((N,), -11.0),
            "lowest": torch.full((N,), -40.0),
            "levels": torch.tensor([-2.0, -11.0, -40.0])[j // 128 % 3],
            "levels back": torch.tensor([-40.0, -11.0, -2.0])[j // 128 % 3]}[pattern]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [5.0, 20.0, 29.0, 30.0, 50.0])
@pytest.mark.parametrize("pattern", ["zero", "against", "turning"])
@pytest.mark.parametrize("B, H, Hkv, N, kind", [(1, 2, 1, 1024, "full"), (4, 40, 40, 256, "full"), (1, 2, 1, 600, "prefix")])
def test_no_product_above_zero(B, H, Hkv, N, kind, pattern, cap, d):
    """Queries of zeros, and queries that all or most keys point away from: in few items, which shares
    cut, and in many."""
    both_ways(directed(B, H, Hkv, N, d, caps_of(pattern, N), cap), kind, cap, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [5.0, 20.0, 29.0, 30.0, 50.0])
@pytest.mark.parametrize("pattern", ["zero", "against", "turning"])
@pytest.mark.parametrize("T", [1, 17, 60, 150])
def test_no_product_above_zero_over_pages(T, pattern, cap, d):
    """A few rows, one row tile and pairs of them."""
    over_pages(T, pattern, cap, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [8.0, 30.0, 50.0])
@pytest.mark.parametrize("pattern", ["low", "lowest", "levels", "levels back"])
@pytest.mark.parametrize("N, kind", [(100, "causal"), (700, "causal"), (700, "docs"), (384, "full"), (700, "random")])
def test_products_many_caps_below_zero(N, kind, pattern, cap, d):
    """Rows that see nothing but products of -2, -11 and -40 caps: the scores are all about -cap."""
    both_ways(directed(1, 4, 2, N, d, caps_of(pattern, N), cap), kind, cap, d)


@pytest.mark.parametrize("cap", [30.0, 50.0])
@pytest.mark.parametrize("kind", ["causal", "docs", "random"])
def test_a_few_rows_of_low_products(kind, cap):
    """Rows 0, 37, 74, ... see products of -15 caps alone, their neighbours ordinary ones."""
    d, N = 128, 500
    q, k, v, do = directed(1, 4, 2, N, d, caps_of("low", N), cap)
    low = q[:, :, ::37] * (15 / 11)
    q = (randn(3, 1, 4, N, d) * 4).cuda()
    q[:, :, ::37] = low
    both_ways((q, k, v, do), kind, cap, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [5.0, 30.0, 50.0])
@pytest.mark.parametrize("pattern", ["low", "lowest", "levels"])
@pytest.mark.parametrize("T", [1, 17, 60, 150])
def test_products_many_caps_below_zero_over_pages(T, pattern, cap, d):
    over_pages(T, pattern, cap, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap, slope", [(30.0, 1.0), (30.0, 0.5), (5.0, 0.25), (5.0, 2.0), (0.0, 1.0)])
@pytest.mark.parametrize("seen", ["far", "far documents", "near"])
def test_hidden_keys_much_nearer_than_the_seen_ones(seen, cap, slope, d):
    """Rows that see far keys alone, in tiles whose other rows see near ones: without its mask the bias would
    make a hidden pair weigh more than fp32 holds.  (near: a bias that grows, and hidden keys that are far.)"""
    N = 2048 if slope < 1 else 512
    i = torch.arange(N, dtype=torch.int32)
    even = i % 2 == 0
    if seen == "far":
        begin, end = torch.where(even, 0, N // 2), torch.where(even, 10, 3 * N // 4)
    elif seen == "far documents":
        begin, end = torch.zeros_like(i), torch.where(even, 10, N)
    else:
        begin, end = torch.where(even, N - 140, N - 256), torch.where(even, N - 120, N)
        slope = -slope
    slopes = torch.tensor([slope, slope / 2, 0.0, -slope / 8])
    x = inputs(1, 4, 2, N, d, cap, 41)
    both_ways([t.cuda() for t in x], None, cap, d, slopes, (begin.int()[None], end.int()[None]))


@pytest.mark.parametrize("cap", [1000.0, 16384.0])
@pytest.mark.parametrize("slopes", [False, True])
def test_small_scores_under_a_large_cap(slopes, cap):
    """The tanh's error, 2^-21 of the cap, is what the bounds count: in all forms, of scores up to 20 or so."""
    d, H = 128, 4
    sl = slopes_of(H, slopes)
    for kind, N in (("causal", 700), ("docs", 300), ("full", 256)):
        both_ways([x.cuda() for x in inputs(1, H, 2, N, d, cap, 51)], kind, cap, d, sl)
    lens, size, scale = [700, 385], 32, 1 / math.sqrt(d)
    for T in (1, 17, 60, 150):
        table, count = tables(lens, [T] * 2, size, -(-(max(lens) + T) // size), 1)
        kp, vp = pool(1, count, 2, size, d, "tokens"), pool(2, count, 2, size, d, "heads")
        q = (randn(3, 2, H, T, d) * 4).cuda()
        o, lse = fa.paged_attention_forward(q, kp, vp, table.cuda(), torch.tensor(lens, **I32).cuda(), scale, cap=cap,
                                            slopes=None if sl is None else sl.cuda())
        check_paged(q, kp, vp, table, o, lse, scale, lens, [T] * 2, 0, cap, sl)
