"""The span and paged kernels' forms side by side and at their borders: waits that run
out, other streams, rows on either side of a form's limit, caps on either side of the
polynomial's range.  Bounds as in test_span_gpu."""

import math

import numpy as np
import pytest
import torch

from exact_tiled_attention_08_gb300 import fa
from test_paged_gpu import check_paged, pool, tables
from test_span_gpu import H2, check_bwd, check_fwd, inputs, masks, randn, slopes_of

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32)
BUSY = 40_000_000  # cycles: some 20 ms


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_tiled_attention_08_gb300.build import build_library

    build_library()
    fa.load_library()
    yield
    fa.fa_debug_stall(False)
    fa.fa_set_wait_limit_ns(0)


def span_call(N, cap=0.0, Hkv=2):
    q, k, v, do = (x.cuda() for x in inputs(2, 4, Hkv, N, 128, cap, N))
    begin, end, causal = masks("docs", 2, N, N)
    args = dict(key_begin=begin.cuda(), key_end=end.cuda(), causal=causal, cap=cap)
    return q, k, v, do, args, (begin, end, causal, 0, cap, None)


def paged_call(B, H, Hkv, T, lens, size=16, d=128, width=None):
    table, count = tables(lens, [T] * B, size, width or -(-(max(lens) + T) // size), 1)
    kp, vp = pool(1, count, Hkv, size, d, "tokens"), pool(2, count, Hkv, size, d, "heads")
    return randn(3, B, H, T, d).cuda(), kp, vp, table, torch.tensor(lens, **I32).cuda()


def calls():
    """Every form of the kernels, as name: (call, check of what it returns)."""
    made = {}
    for name, N in (("pair", 400), ("one tile", 100), ("few rows", 20)):
        q, k, v, do, args, ref = span_call(N)
        made["span " + name] = (lambda q=q, k=k, v=v, args=args, **kw: fa.span_attention_forward(q, k, v, 0.1, **args, **kw),
                                lambda got, q=q, k=k, v=v, ref=ref: check_fwd(q, k, v, *got, 0.1, *ref))
    q, k, v, do, args, ref = span_call(400, 20.0)
    o, lse = fa.span_attention_forward(q, k, v, 0.1, **args)
    made["span backward"] = (
        lambda q=q, k=k, v=v, do=do, o=o, lse=lse, args=args, **kw: fa.span_attention_backward(q, k, v, o, do, lse, 0.1, **args,
                                                                                               **kw),
        lambda got, q=q, k=k, v=v, do=do, o=o, lse=lse, ref=ref: check_bwd(q, k, v, o, do, lse, got, 0.1, *ref))
    for name, case in (("paged pair", (2, 8, 2, 70, [100, 900])), ("paged one tile", (2, 8, 2, 10, [100, 900])),
                       ("paged few rows", (20, 8, 2, 1, [50 * i for i in range(20)])),
                       ("paged cluster", (1, 8, 2, 2, [1500]))):
        B, H, Hkv, T, lens = case
        q, kp, vp, table, dl = paged_call(*case)
        made[name] = (
            lambda q=q, kp=kp, vp=vp, table=table, dl=dl, **kw: fa.paged_attention_forward(q, kp, vp, table.cuda(), dl, 0.1, **kw),
            lambda got, q=q, kp=kp, vp=vp, table=table, lens=lens, T=T, B=B: check_paged(
                q, kp, vp, table, *got, 0.1, lens, [T] * B, 0, 0.0, None))
    return made


NAMES = ["span pair", "span one tile", "span few rows", "span backward", "paged pair", "paged one tile", "paged few rows",
         "paged cluster"]


@pytest.mark.parametrize("name", NAMES)
def test_waits_that_run_out_are_reported(name):
    """The issuing thread stalls: the kernels stop, the status says so, and the next call is right."""
    call, check = calls()[name]
    check(call())
    assert fa.fa_check_device_status() == fa.FA_OK
    try:
        fa.fa_set_wait_limit_ns(1_000_000)
        fa.fa_debug_stall(True)
        call(check_status=False)
        assert fa.fa_check_device_status() == fa.FA_ERR_TIMEOUT
        with pytest.raises(fa.FaError) as err:
            call()
        assert err.value.status == fa.FA_ERR_TIMEOUT
    finally:
        fa.fa_debug_stall(False)
        fa.fa_set_wait_limit_ns(0)
    assert fa.fa_check_device_status() == fa.FA_OK
    check(call())


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_call_on_another_stream_than_the_current_one(name, raw):
    call, check = calls()[name]
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    got = call(stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    check(got)
    for a, b in list(zip(got, want))[1 if name == "span backward" else 0:]:  # (dQ is summed in any order)
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 1), (1, 16), (15, 1), (16, 1), (17, 1), (4, 8), (33, 1), (3, 11), (128, 1), (43, 3)])
def test_rows_on_either_side_of_a_form(T, G, d):
    """1 to 129 rows that share a key/value head: 16, 32 and 128 are the forms' limits."""
    lens = [700, 3]
    q, kp, vp, table, dl = paged_call(2, 2 * G, 2, T, lens, 32, d)
    slopes = slopes_of(2 * G, True)
    for window, cap, sl in ((0, 0.0, None), (90, 10.0, slopes), (0, 40.0, None), (0, 0.0, slopes)):
        o, lse = fa.paged_attention_forward(q, kp, vp, table.cuda(), dl, 0.2, window=window, cap=cap,
                                            slopes=None if sl is None else sl.cuda())
        check_paged(q, kp, vp, table, o, lse, 0.2, lens, [T] * 2, window, cap, sl)


@pytest.mark.parametrize("items", [7, 15, 16, 36, 37, 76, 77])
@pytest.mark.parametrize("n", [300, 9000])
def test_on_either_side_of_the_cluster_rule(items, n):
    """One request whose heads are the items: one more of them than the device holds clusters."""
    q, kp, vp, table, dl = paged_call(1, 2 * items, items, 1, [n], 64, 64)
    o, lse = fa.paged_attention_forward(q, kp, vp, table.cuda(), dl, 0.125)
    check_paged(q, kp, vp, table, o, lse, 0.125, [n], [1], 0, 0.0, None)


@pytest.mark.parametrize("width", [94, 1000, 40000])
def test_pages_that_a_request_may_have(width):
    """A short request in a table of any width: the number of CTAs that share its keys changes."""
    q, kp, vp, table, dl = paged_call(1, 8, 2, 1, [1490], 16, 128, width)
    o, lse = fa.paged_attention_forward(q, kp, vp, table.cuda(), dl, 0.1)
    check_paged(q, kp, vp, table, o, lse, 0.1, [1490], [1], 0, 0.0, None)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [5.0, 29.0, 30.0, 50.0, 1e4])
@pytest.mark.parametrize("kind", ["causal", "random", "docs"])
def test_products_around_the_range_of_the_polynomial(kind, cap, d):
    """Rows whose products lie below, in and above what the polynomial takes, on either side of 0: scores of
    +-0.1, 0.5, 1 and 2 caps, rows that have only negative ones, and rows of one large one."""
    B, H, Hkv, N = 1, 4, 2, 400
    q, k, v, do = (x.cuda() for x in inputs(B, H, Hkv, N, d, 0.0, 21))
    size = torch.tensor([0.1, 0.5, 1.0, 2.0], device="cuda").repeat_interleave(50).repeat(2)
    q = (q.float() * size[None, None, :, None] * cap / 3).bfloat16()  # (products of norm d, times scale d^-1/2: about 1)
    k[:, :, 200:] = -k[:, :, :1]          # half of the keys point away from the first
    q[:, :, ::7] = (k[:, :, :1].float() * cap / 8).bfloat16().repeat_interleave(2, 1)  # and some queries to it
    begin, end, causal = masks(kind, B, N, 5)
    args = dict(key_begin=None if begin is None else begin.cuda(), key_end=None if end is None else end.cuda(), causal=causal)
    scale = 1 / math.sqrt(d)
    o, lse = fa.span_attention_forward(q, k, v, scale, cap=cap, **args)
    check_fwd(q, k, v, o, lse, scale, begin, end, causal, 0, cap, None)
    if cap < 1e3:  # (a score's own rounding, 2^-24 of it and more, would be all of P at 1e4)
        grads = fa.span_attention_backward(q, k, v, o, do, lse, scale, cap=cap, **args)
        check_bwd(q, k, v, o, do, lse, grads, scale, begin, end, causal, 0, cap, None)


def test_what_is_hidden_has_no_say_in_the_cap():
    """Hidden products that are huge, infinite or NaN leave the others' bits as they are.  (Rows 250 and on see
    them, and a warp chooses how to cap for its 32 rows together: rows 224 to 249 stay within the bounds.)"""
    B, H, Hkv, N = 1, 4, 2, 300
    for cap in (10.0, 50.0):
        q, k, v, _ = (x.cuda() for x in inputs(B, H, Hkv, N, 128, cap, 30))
        want = None
        for fill in (0.0, 1e30, float("inf"), float("nan")):
            k[:, :, 250:] = fill
            o, lse = fa.span_attention_forward(q, k, v, 0.1, causal=True, cap=cap)
            got = o[:, :, :224], lse[:, :, :224]
            want = want or got
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (cap, fill)
            cut = [x[:, :, :250].contiguous() for x in (q, k, v)]
            check_fwd(*cut, o[:, :, :250], lse[:, :, :250], 0.1, None, None, True, 0, cap, None)


@pytest.mark.parametrize("case", [
    (1, 160, 160, 200, "full", 0),        # a last round that is not full
    (2, 130, 130, 300, "docs", 0),
    (1, 1, 1, 9000, "causal", 0),         # few long items: shares
    (1, 3, 3, 5000, "full", 700),
    (40, 8, 8, 257, "docs", 0),           # more entries than there are threads to sort them
    (200, 8, 4, 300, "prefix", 0),
    (1, 700, 700, 260, "causal", 0),
    (12, 64, 64, 900, "full", 300),       # more than 32 items a CTA: head by head
    (70, 80, 80, 260, "causal", 0),       # the same, entry by entry
])
def test_ways_of_handing_out_items(case):
    """Every way in which the CTAs divide the items, each head against fp32."""
    B, H, Hkv, N, kind, window = case
    d = 64
    q, k, v, _ = (x.cuda() for x in inputs(B, H, Hkv, N, d, 0.0, 3))
    begin, end, causal = masks(kind, B, N, 4)
    dev = [None if x is None else x.cuda() for x in (begin, end)]
    scale = 0.125
    o, lse = fa.span_attention_forward(q, k, v, scale, *dev, causal=causal, window=window)
    check_fwd(q, k, v, o, lse, scale, begin, end, causal, window, 0.0, None)
    i = torch.arange(N, device="cuda")
    for b in range(B):
        seen = torch.ones((N, N), dtype=torch.bool, device="cuda")
        if dev[0] is not None:
            seen &= i[None] >= dev[0][b][:, None]
        if dev[1] is not None:
            seen &= i[None] < dev[1][b][:, None]
        if causal:
            seen &= i[None] <= i[:, None]
        if window:
            seen &= (i[:, None] - i[None]).abs() < window
        s = torch.matmul(q[b].float(), k[b].float().repeat_interleave(H // Hkv, 0).transpose(-1, -2)) * scale
        s = s.masked_fill(~seen, -math.inf)
        ref = torch.logsumexp(s, -1)
        p = torch.exp(s - ref.clamp(min=-1e30)[..., None])
        want = torch.matmul(p, v[b].float().repeat_interleave(H // Hkv, 0))
        # (both sides fp32 but for P and O: within 3 half steps of the largest value)
        assert (o[b].float() - want).abs().max() <= 4 * H2 * v.float().abs().max()
        live = ref > -math.inf
        assert torch.equal(live, lse[b] > -math.inf) and (lse[b][live] - ref[live]).abs().max() <= 1e-3


@pytest.mark.parametrize("case", [(1, 8, 1, 1000, "causal", 0), (1, 2, 2, 2500, "docs", 0), (3, 4, 4, 600, "full", 100),
                                  (1, 2, 1, 129, "random", 0), (9, 40, 40, 130, "prefix", 0), (2, 16, 4, 1000, "causal", 0)])
def test_ways_of_cutting_the_backward(case):
    """Items that are whole and items in runs; twice, with the same dK and dV."""
    B, H, Hkv, N, kind, window = case
    for d in (64, 128):
        q, k, v, do = (x.cuda() for x in inputs(B, H, Hkv, N, d, 0.0, 4))
        begin, end, causal = masks(kind, B, N, 6)
        args = dict(key_begin=None if begin is None else begin.cuda(), key_end=None if end is None else end.cuda(), causal=causal,
                    window=window)
        o, lse = fa.span_attention_forward(q, k, v, 0.1, **args)
        grads = fa.span_attention_backward(q, k, v, o, do, lse, 0.1, **args)
        check_bwd(q, k, v, o, do, lse, grads, 0.1, begin, end, causal, window, 0.0, None)
        again = fa.span_attention_backward(q, k, v, o, do, lse, 0.1, **args)
        assert torch.equal(grads[1], again[1]) and torch.equal(grads[2], again[2])


def test_unaligned_rows_of_masks_and_outputs():
    """Masks that start on any element; outputs on 16-byte boundaries that are not 32-byte ones."""
    B, H, Hkv, N, d = 2, 4, 2, 300, 128
    q, k, v, do = (x.cuda() for x in inputs(B, H, Hkv, N, d, 0.0, 15))
    begin, end, _ = masks("docs", B, N, 2)

    def shifted(x, by):
        memory = torch.empty((x.numel() + by,), dtype=x.dtype, device="cuda")
        y = memory[by:].view(x.shape)
        y.copy_(x)
        return y

    b, e = shifted(begin.cuda(), 1), shifted(end.cuda(), 3)
    o, lse = shifted(torch.empty_like(q), 8), torch.empty((B, H, N), device="cuda")
    g = [shifted(torch.empty_like(x), 8) for x in (q, k, v)]
    wf = torch.empty(fa.fa_span_fwd_workspace_bytes(B, H, Hkv, N, d) + 16, dtype=torch.uint8, device="cuda")[16:]
    wb = torch.empty(fa.fa_span_bwd_workspace_bytes(B, H, Hkv, N, d) + 16, dtype=torch.uint8, device="cuda")[16:]
    fa.fa_span_fwd(q, k, v, b, e, o, lse, wf, 0.1, causal=True)
    fa.fa_span_bwd(q, k, v, b, e, o, do, lse, *g, wb, 0.1, causal=True)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_fwd(q, k, v, o, lse, 0.1, begin, end, True, 0, 0.0, None)
    check_bwd(q, k, v, o, do, lse, g, 0.1, begin, end, True, 0, 0.0, None)


def test_a_training_step():
    """Norm and rotation, attention to packed documents with a cap, its gradients and the rotation's, on one stream
    without a synchronisation: each part by its bounds, and the projection's gradient against differences of the
    oracle."""
    from oracle.cross import rope_bwd_ref, rope_ref
    from oracle.span import span_attention_ref
    from test_span_gpu import host, seen_of

    B, N, H, Hkv, d, cap, scale = 1, 260, 4, 2, 64, 20.0, 0.3
    rows, do = randn(1, B, N, H + 2 * Hkv, d), randn(2, B, H, N, d)
    begin, end, _ = masks("docs", B, N, 8)
    x = rows.cuda()
    q, k, v = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
    freq = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    w = torch.ones((d,), device="cuda")
    qr = torch.empty((B, H, N, d), dtype=torch.bfloat16, device="cuda")
    kr, vr = (torch.empty((B, Hkv, N, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.fa_rope_fwd(q, k, v, w, w, freq, None, None, qr, kr, vr, eps=1e-6)
    args = dict(key_begin=begin.cuda(), key_end=end.cuda(), causal=True, cap=cap, check_status=False)
    o, lse = fa.span_attention_forward(qr, kr, vr, scale, **args)
    g = fa.span_attention_backward(qr, kr, vr, o, do.cuda(), lse, scale, **args)
    dx = torch.empty_like(x)
    dw = [torch.empty((d,), device="cuda") for _ in range(2)]
    ws = torch.empty(fa.fa_rope_bwd_workspace_bytes(B, H, Hkv, N, d), dtype=torch.uint8, device="cuda")
    fa.fa_rope_bwd(q, k, w, w, freq, None, *g, dx[:, :, :H], dx[:, :, H:H + Hkv], dx[:, :, H + Hkv:], *dw, ws, eps=1e-6)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_bwd(qr, kr, vr, o, do, lse, g, scale, begin, end, True, 0, cap, None)
    seen, one = seen_of(begin, end, True, 0, 0, N), np.ones(d)
    f, pos = freq.cpu().numpy(), np.arange(N)
    for h in range(H):  # the rotation's part, from the gradients at hand
        ref, _ = rope_bwd_ref(host(rows[0, :, h]), one, f, pos, host(g[0][0, h]), 1e-6)
        assert np.abs(host(dx[0, :, h]) - ref).max() <= H2 * np.abs(ref).max() + 1e-5 * np.abs(ref).max()
    # a direction of the first head's rows: the oracle's step through all of it
    x0 = host(rows[0, :, 0])
    u = np.random.default_rng(0).standard_normal(x0.shape)

    def step(t):
        qn = rope_ref(x0 + t * u, one, f, pos, 1e-6)
        ref = span_attention_ref(qn, host(kr[0, 0]), host(vr[0, 0]), scale, seen, cap)
        return (ref[0] * host(do[0, 0])).sum()

    got = host(dx[0, :, 0])
    # (as in test_span_gpu's differences, and the rounding of the rotated rows to bf16, relative to the scores' size)
    assert abs((got * u).sum() - (step(1e-4) - step(-1e-4)) / 2e-4) <= 64 * H2 * np.linalg.norm(got)


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last group of heads comes out as it does alone."""
    B, H, Hkv, N, d, window = 1, 300, 30, 60000, 128, 300
    assert B * H * N * d > 2 ** 31
    g = torch.Generator("cuda").manual_seed(1)
    q, k, v, do = (torch.randn((B, h, N, d), generator=g, device="cuda", dtype=torch.bfloat16) for h in (H, Hkv, Hkv, H))
    o, lse = fa.span_attention_forward(q, k, v, 0.1, causal=True, window=window)
    grads = fa.span_attention_backward(q, k, v, o, do, lse, 0.1, causal=True, window=window)
    G = H // Hkv
    one = [x[:, -n:].contiguous() for x, n in ((q, G), (k, 1), (v, 1), (do, G))]
    p, ple = fa.span_attention_forward(*one[:3], 0.1, causal=True, window=window)
    alone = fa.span_attention_backward(*one[:3], p, one[3], ple, 0.1, causal=True, window=window)
    # (alone, items may be cut into other parts, which are added up in fp32: a bf16 step of the largest)
    for x, y in zip((o[:, -G:], grads[0][:, -G:], grads[1][:, -1:], grads[2][:, -1:]), (p, *alone)):
        assert float((x.float() - y.float()).abs().max()) <= 2 ** -7 * float(y.float().abs().max())
    assert float((lse[:, -G:] - ple).abs().max()) <= 1e-4
