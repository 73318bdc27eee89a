"""Attention of chunks over a cache in pages (fa_paged_fwd), and rotation into pages
(fa_rope_paged_fwd), against the fp64 oracle.  Bounds of the attention as in
test_span_gpu, of the rotation as in test_rope_gpu: what is written is rounded once,
H = 2^-8 of the value, from fp32 arithmetic (1e-6 of the row's largest value).
"""

import math

import numpy as np
import pytest
import torch

from exact_tiled_attention_08_gb300 import fa
from oracle.cross import rope_ref
from oracle.span import gather_pages, span_attention_ref, span_seen
from test_span_gpu import check_rows, host, randn, slopes_of

pytestmark = pytest.mark.gpu

H2 = 2.0 ** -8
I32 = dict(dtype=torch.int32)


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_tiled_attention_08_gb300.build import build_library

    build_library()
    fa.load_library()
    assert torch.cuda.is_available()


def pool(seed, count, Hkv, size, d, layout):
    """Pages [count, Hkv, size, d] of a cache in one of three layouts."""
    if layout == "heads":
        return randn(seed, count, Hkv, size, d).cuda()
    if layout == "tokens":
        return randn(seed, count, size, Hkv, d).cuda().transpose(1, 2)
    return randn(seed, count, 2, size, Hkv, d + 64).cuda()[:, 1, :, :, :d].transpose(1, 2)  # beside others


def tables(lens, chunks, size, width, seed, count=None):
    """Page numbers in any order, garbage behind the pages in use."""
    g = np.random.default_rng(seed)
    need = [-(-(n + c) // size) for n, c in zip(lens, chunks)]
    count = sum(need) + 3 if count is None else count
    order = g.permutation(count)
    table = g.choice([-1, 2 ** 31 - 1, -2 ** 31, count], (len(lens), width)).astype(np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table.astype(np.int32)), count


def check_paged(q, kp, vp, table, o, lse, scale, lens, chunks, window, cap, slopes, fill=7.0, most=8):
    B, H, T, _ = q.shape
    Hkv, size = kp.shape[1:3]
    every = [(b, h) for b in range(B) for h in range(H)]
    some = every if len(every) <= most else [every[i * (len(every) - 1) // (most - 1)] for i in range(most)]
    for b, h in some:
        n, c = lens[b], chunks[b]
        j = h // (H // Hkv)
        k, v = (gather_pages(host(x[:, j]), table[b].tolist(), n + c) for x in (kp, vp))
        seen = span_seen(c, causal=True, window=window, first=n, keys=n + c)
        if c:
            ref = span_attention_ref(host(q[b, h, :c]), k, v, scale, seen, cap,
                                     0.0 if slopes is None else float(slopes[h]), n)
            check_rows(host(o[b, h, :c]), host(lse[b, h, :c]), ref, (b, h))
    for b in range(B):  # rows of tokens that are not there
        assert (o[b, :, chunks[b]:] == fill).all() and (lse[b, :, chunks[b]:] == fill).all()


CASES = [
    # B, H, Hkv, T, page size, lens, chunks, window, cap, slopes, layout, entries more than needed
    (1, 1, 1, 1, 16, [0], None, 0, 0.0, False, "heads", 0),
    (1, 8, 2, 1, 16, [299], None, 0, 50.0, False, "tokens", 3),
    (3, 4, 2, 1, 32, [0, 127, 128], None, 0, 0.0, True, "heads", 1),
    (2, 4, 4, 5, 16, [126, 255], [5, 3], 0, 0.0, False, "beside", 0),
    (3, 2, 1, 64, 64, [0, 100, 336], [64, 0, 63], 50, 0.0, False, "tokens", 2),
    (1, 8, 1, 40, 128, [900], [39], 0, 20.0, True, "heads", 0),
    (2, 3, 1, 200, 256, [250, 299], [200, 150], 0, 0.0, False, "tokens", 1),
    (2, 16, 4, 129, 512, [0, 700], None, 200, 30.0, False, "heads", 0),
    (4, 16, 8, 7, 16, [4990, 2000, 0, 129], [7, 7, 2, 7], 0, 0.0, False, "heads", 5),
    (1, 2, 1, 3, 32, [29000], None, 0, 0.0, False, "tokens", 0),
    (1, 2, 1, 1, 16, [20000], None, 130, 0.0, True, "heads", 0),
    (40, 16, 8, 2, 16, list(range(0, 280, 7)), None, 0, 0.0, False, "heads", 0),
    (1, 2, 2, 700, 64, [0], None, 0, 0.0, False, "heads", 0),
    (2, 4, 2, 600, 32, [513, 0], [600, 257], 256, 0.0, True, "tokens", 0),
    (1, 32, 8, 1, 16, [1907], None, 0, 0.0, False, "tokens", 0),
    (1, 4, 4, 1000, 16, [3], None, 0, 15.0, False, "heads", 0),
    (20, 16, 8, 3, 64, [3990 - 7 * i for i in range(20)], None, 0, 0.0, False, "heads", 0),
    (6, 40, 5, 130, 128, [0, 5, 900, 128, 127, 300], [130, 1, 0, 129, 128, 2], 0, 0.0, False, "heads", 0),
    (2, 8, 8, 3, 16, [0, 60], [0, 0], 0, 0.0, False, "heads", 1),
]


def chunks_of(case):
    return [case[3]] * case[0] if case[6] is None else list(case[6])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CASES)
def test_forward(case, d):
    B, H, Hkv, T, size, lens, some, window, cap, slopes, layout, more = case
    chunks = chunks_of(case)
    width = max(1, max(-(-(n + c) // size) for n, c in zip(lens, chunks))) + more
    table, count = tables(lens, chunks, size, width, T)
    kp, vp = pool(T, count, Hkv, size, d, layout), pool(T + 1, count, Hkv, size, d, layout)
    for b, (n, c) in enumerate(zip(lens, chunks)):  # behind a request's last token, and in pages of nobody
        if (n + c) % size:
            page = int(table[b, (n + c) // size])
            kp[page, :, (n + c) % size:] = float("nan")
            vp[page, :, (n + c) % size:] = float("inf")
    used = {int(x) for b, (n, c) in enumerate(zip(lens, chunks)) for x in table[b, :-(-(n + c) // size)]}
    for page in set(range(count)) - used:
        kp[page], vp[page] = float("nan"), float("nan")
    q = randn(T + 2, B, H, T, d).cuda() * (4 if cap else 1)
    sl = slopes_of(H, slopes)
    scale = 1 / math.sqrt(d)
    o, lse = torch.full_like(q, 7.0), torch.full((B, H, T), 7.0, device="cuda")
    n = fa.fa_paged_fwd_workspace_bytes(B, H, Hkv, T, width * size, d)
    memory = torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda")
    args = (q, kp, vp, table.cuda(), torch.tensor(lens, **I32).cuda(),
            None if some is None else torch.tensor(some, **I32).cuda())
    for _ in range(2):
        fa.fa_paged_fwd(*args, o, lse, memory[:n], scale, window=window, cap=cap,
                        slopes=None if sl is None else sl.cuda())
        assert fa.fa_check_device_status() == fa.FA_OK
        assert (memory[n:] == 255).all()
        check_paged(q, kp, vp, table, o, lse, scale, lens, chunks, window, cap, sl)
        first, o, lse = (o, lse), torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    fa.fa_paged_fwd(*args, o, lse, memory[:n], scale, window=window, cap=cap, slopes=None if sl is None else sl.cuda())
    assert torch.equal(first[0], o) and torch.equal(first[1], lse)


def test_chunks_that_do_not_fit_and_lengths_outside_the_pages():
    """Three entries of 16 tokens: at most 48, whatever the lengths say."""
    table = torch.arange(9, **I32).reshape(3, 3)
    kp, vp = pool(1, 9, 2, 16, 64, "heads"), pool(2, 9, 2, 16, 64, "heads")
    q = randn(3, 3, 4, 8, 64).cuda()
    o, lse = torch.full_like(q, 7.0), torch.full((3, 4, 8), 7.0, device="cuda")
    ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(3, 4, 2, 8, 48, 64), dtype=torch.uint8, device="cuda")
    fa.fa_paged_fwd(q, kp, vp, table.cuda(), torch.tensor([43, 2 ** 31 - 1, -5], **I32).cuda(),
                    torch.tensor([8, 8, 2 ** 31 - 1], **I32).cuda(), o, lse, ws, 0.125)
    check_paged(q, kp, vp, table, o, lse, 0.125, [43, 48, 0], [5, 0, 8], 0, 0.0, None)


def test_pages_outside_the_pool_are_zeros():
    """Bad page numbers among those in use: their keys score 0 and their values are 0."""
    size, lens, chunks = 16, [100, 37], [4, 4]
    table, count = tables(lens, chunks, size, 8, 5)
    for b, i, page in ((0, 0, -1), (0, 3, 2 ** 31 - 1), (0, 5, count), (1, 1, -2 ** 31)):
        table[b, i] = page
    for size_now, fold in ((16, 1), (256, 16)):
        kp, vp = pool(1, count, 2, size_now, 128, "heads"), pool(2, count, 2, size_now, 128, "tokens")
        lens_now, chunks_now = [n * fold for n in lens], chunks
        q = randn(3, 2, 4, 4, 128).cuda()
        o, lse = fa.paged_attention_forward(q, kp, vp, table.cuda(), torch.tensor(lens_now, **I32).cuda(), 0.1)
        check_paged(q, kp, vp, table, o, lse, 0.1, lens_now, chunks_now, 0, 0.0, None)


def test_shared_pages():
    """Two requests that share their first pages, and one page many times in one request."""
    kp, vp = pool(1, 6, 2, 32, 64, "heads"), pool(2, 6, 2, 32, 64, "heads")
    table = torch.tensor([[0, 1, 2, 2], [0, 1, 3, 5], [4, 4, 4, 4]], **I32)
    q = randn(3, 3, 4, 2, 64).cuda()
    lens = [125, 70, 100]
    o, lse = fa.paged_attention_forward(q, kp, vp, table.cuda(), torch.tensor(lens, **I32).cuda(), 0.1)
    check_paged(q, kp, vp, table, o, lse, 0.1, lens, [2, 2, 2], 0, 0.0, None)


def test_windows_leave_freed_pages_alone():
    """Entries of pages in front of every query's window are never used."""
    size, n, T, window = 16, 1000, 8, 100
    table, count = tables([n], [T], size, 63, 4)
    kp, vp = pool(1, count, 2, size, 128, "heads"), pool(2, count, 2, size, 128, "heads")
    q = randn(3, 1, 8, T, 128).cuda()
    lens = torch.tensor([n], **I32).cuda()
    want = fa.paged_attention_forward(q, kp, vp, table.cuda(), lens, 0.1, window=window)
    first = (n - window + 1) // size
    bad = int(table[0, 0])
    kp[bad], vp[bad] = float("nan"), float("nan")
    freed = table.clone()
    for value in (-1, bad, 2 ** 31 - 1):
        freed[0, :first] = value
        got = fa.paged_attention_forward(q, kp, vp, freed.cuda(), lens, 0.1, window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), value


def test_offsets_past_32_bits():
    """Pools of more than 2^31 elements, pages at both ends."""
    count, Hkv, size, d = 70000, 2, 128, 128
    kp = torch.zeros((count, Hkv, size, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    kk, vv = randn(1, 4, Hkv, size, d).cuda(), randn(2, 4, Hkv, size, d).cuda()
    for i, page in enumerate((0, count - 1, 66000, 3)):
        kp[page], vp[page] = kk[i], vv[i]
    q = randn(3, 1, 4, 5, d).cuda()
    lens = torch.tensor([500], **I32).cuda()
    far = fa.paged_attention_forward(q, kp, vp, torch.tensor([[0, count - 1, 66000, 3]], **I32).cuda(), lens, 0.1)
    near = fa.paged_attention_forward(q, kk, vv, torch.arange(4, **I32)[None].cuda(), lens, 0.1)
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
    # rotation into the same pages
    rows = randn(4, 1, 5, Hkv, d).cuda()
    table = torch.tensor([[0, count - 1, 66000, 3]], **I32).cuda()
    fa.fa_rope_paged_fwd(None, rows, rows, None, None, None, None, table, torch.tensor([254], **I32).cuda(), None, None,
                         kp, vp)
    assert torch.equal(kp[count - 1, :, 126:], rows[0, :2].transpose(0, 1))
    assert torch.equal(vp[66000, :, :3], rows[0, 2:].transpose(0, 1))


def test_replayed_graph_and_other_stream():
    """A captured chunk, replayed with other lengths, tables and pages, on another stream too."""
    B, H, Hkv, T, size, d, width = 3, 8, 2, 20, 32, 64, 30
    q = randn(1, B, H, T, d).cuda()
    count = 3 * width
    kp, vp = pool(2, count, Hkv, size, d, "tokens"), pool(3, count, Hkv, size, d, "tokens")
    lens, chunks = [900, 0, 77], [20, 3, 11]
    table, _ = tables(lens, chunks, size, width, 1, count)
    dt, dl, dc = table.cuda(), torch.tensor(lens, **I32).cuda(), torch.tensor(chunks, **I32).cuda()
    o, lse = torch.full_like(q, 7.0), torch.full((B, H, T), 7.0, device="cuda")
    ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(B, H, Hkv, T, width * size, d), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        fa.fa_paged_fwd(q, kp, vp, dt, dl, dc, o, lse, ws, 0.125, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.synchronize()
    check_paged(q, kp, vp, table, o, lse, 0.125, lens, chunks, 0, 0.0, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, lens, chunks in ((2, [3, 940, 128], [20, 20, 0]), (3, [0, 0, 500], [1, 20, 20])):
        table, _ = tables(lens, chunks, size, width, seed, count)
        dt.copy_(table), dl.copy_(torch.tensor(lens, **I32)), dc.copy_(torch.tensor(chunks, **I32))
        o.fill_(7.0), lse.fill_(7.0)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_check_device_status() == fa.FA_OK
        check_paged(q, kp, vp, table, o, lse, 0.125, lens, chunks, 0, 0.0, None)


ROPE = [
    # B, N, H, Hkv, page size, lens, chunks, rotated part, norm, interleaved, layout, positions
    (1, 1, 1, 1, 16, [0], None, 1.0, False, False, "heads", False),
    (3, 1, 8, 2, 16, [15, 16, 4000], None, 1.0, False, False, "tokens", False),
    (2, 40, 6, 3, 32, [31, 0], [40, 17], 0.5, True, True, "beside", False),
    (2, 300, 4, 2, 128, [100, 700], [300, 0], 1.0, True, False, "heads", True),
    (1, 130, 2, 1, 64, [1], None, 0.0, True, False, "tokens", False),
    (5, 9, 16, 8, 256, [0, 250, 255, 256, 1000], [9, 9, 1, 8, 9], 1.0, False, True, "heads", False),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", ROPE)
def test_rotation_into_pages(case, d):
    B, N, H, Hkv, size, lens, some, part, norm, inter, layout, positions = case
    chunks = [N] * B if some is None else some
    width = max(-(-(n + c) // size) for n, c in zip(lens, chunks)) + 1
    table, count = tables(lens, chunks, size, width, N)
    kp, vp = pool(N, count, Hkv, size, d, layout), pool(N + 1, count, Hkv, size, d, layout)
    before = kp.clone(), vp.clone()
    rows = randn(N + 2, B, N, H + 2 * Hkv, d).cuda()
    q, k, v = rows[:, :, :H], rows[:, :, H:H + Hkv], rows[:, :, H + Hkv:]
    w = (1 + 0.2 * torch.randn((2, d), generator=torch.Generator().manual_seed(N))) if norm else None
    rot = int(d * part)
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1)) if rot else None
    pos = None
    if positions:
        pos = torch.randint(0, 100000, (B, N), generator=torch.Generator().manual_seed(N), **I32)
    q_out = torch.full((B, H, N, d), 7.0, dtype=torch.bfloat16, device="cuda")
    args = dict(eps=1e-6 if norm else None, factor=1.5, interleaved=inter)
    fa.fa_rope_paged_fwd(q, k, v, None if w is None else w[0].cuda(), None if w is None else w[1].cuda(),
                         None if freq is None else freq.cuda(), None if pos is None else pos.cuda(), table.cuda(),
                         torch.tensor(lens, **I32).cuda(), None if some is None else torch.tensor(some, **I32).cuda(),
                         q_out, kp, vp, **args)
    assert fa.fa_check_device_status() == fa.FA_OK
    wrote = torch.zeros((count, size), dtype=torch.bool, device="cuda")
    for b in range(B):
        n, c = lens[b], chunks[b]
        assert (q_out[b, :, c:] == 7).all()
        if not c:
            continue
        at = np.arange(n, n + c)
        p = at if pos is None else pos[b, :c].numpy()
        f = np.zeros(0) if freq is None else freq.numpy()
        page, row = table[b].numpy()[at // size], at % size
        wrote[page, row] = True
        for x, weight, got in ((q, 0, q_out[b, :, :c]), (k, 1, kp[page, :, row].transpose(0, 1))):
            for h in range(x.shape[2]):
                ref = rope_ref(host(x[b, :c, h]), None if w is None else w[weight].numpy(), f, p,
                               1e-6 if norm else None, 1.5, inter)
                err = np.abs(host(got[h]) - ref)
                assert (err <= H2 * np.abs(ref) + 1e-6 * np.abs(ref).max()).all(), (b, h, err.max())
        assert torch.equal(vp[page, :, row], v[b, :c])
    for now, was in zip((kp, vp), before):  # the other rows
        assert torch.equal(now.transpose(1, 2)[~wrote], was.transpose(1, 2)[~wrote])


def test_rotation_leaves_out_what_has_no_place():
    """Tokens behind the capacity, pages outside the pool, and tensors that are not given."""
    kp, vp = pool(1, 4, 2, 16, 64, "heads"), pool(2, 4, 2, 16, 64, "heads")
    before = kp.clone(), vp.clone()
    rows = randn(3, 2, 20, 2, 64).cuda()
    table = torch.tensor([[3, 0], [-1, 4]], **I32).cuda()
    lens = torch.tensor([20, 0], **I32).cuda()
    fa.fa_rope_paged_fwd(None, rows, rows, None, None, None, None, table, lens, None, None, kp, vp)
    for now, was in zip((kp, vp), before):
        assert torch.equal(now[0, :, 4:], rows[0, :12].transpose(0, 1))
        assert torch.equal(now[0, :, :4], was[0, :, :4]) and torch.equal(now[1:], was[1:])
    # queries alone need no pages
    q_out = torch.full((2, 2, 20, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.fa_rope_paged_fwd(rows, None, None, None, None, None, None, None, None, torch.tensor([20, 3], **I32).cuda(),
                         q_out, None, None)
    assert torch.equal(q_out[0], rows[0].transpose(0, 1)) and torch.equal(q_out[1, :, :3], rows[1, :3].transpose(0, 1))
    assert (q_out[1, :, 3:] == 7).all()


def test_a_prompt_in_chunks_and_then_tokens():
    """A model's layer as it is served: chunks of a prompt are rotated into the pages and attend to them, then
    single tokens; the same layer in one piece through the contiguous rotation and the span attention."""
    B, H, Hkv, d, size, window, cap = 2, 8, 2, 128, 32, 300, 30.0
    total = [500, 333]
    n = max(total)
    rows = randn(1, B, n, H + 2 * Hkv, d).cuda()
    q, k, v = rows[:, :, :H], rows[:, :, H:H + Hkv], rows[:, :, H + Hkv:]
    w = torch.ones((d,), device="cuda")
    freq = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    slopes = slopes_of(H, True).cuda()
    scale = 0.3
    qr = torch.empty((B, H, n, d), dtype=torch.bfloat16, device="cuda")
    kr, vr = (torch.empty((B, Hkv, n, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.fa_rope_fwd(q, k, v, w, w, freq, None, None, qr, kr, vr, eps=1e-6)
    whole, whole_lse = fa.span_attention_forward(qr, kr, vr, scale, causal=True, window=window, cap=cap, slopes=slopes)
    width = -(-n // size)
    table, count = tables(total, [0, 0], size, width, 1)
    kp, vp = (torch.full((count, size, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
              for _ in range(2))
    done = [0, 0]
    for step in [200] * 3 + [1] * 4:
        chunks = [max(0, min(step, t - x - (4 if step > 1 else 0))) for x, t in zip(done, total)]
        T = max(chunks)
        part = torch.zeros((B, T, H + 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")
        for b in range(B):
            part[b, :chunks[b]] = rows[b, done[b]:done[b] + chunks[b]]
        dl, dc = torch.tensor(done, **I32).cuda(), torch.tensor(chunks, **I32).cuda()
        q_out = torch.zeros((B, H, T, d), dtype=torch.bfloat16, device="cuda")
        fa.fa_rope_paged_fwd(part[:, :, :H], part[:, :, H:H + Hkv], part[:, :, H + Hkv:], w, w, freq, None,
                             table.cuda(), dl, dc, q_out, kp, vp, eps=1e-6)
        o, lse = fa.paged_attention_forward(q_out, kp, vp, table.cuda(), dl, scale, chunk_lens=dc, window=window,
                                            cap=cap, slopes=slopes)
        for b in range(B):
            at = slice(done[b], done[b] + chunks[b])
            assert torch.equal(q_out[b, :, :chunks[b]], qr[b, :, at])
            # both sides within the bounds of O: H (A + 2 |O|) with A, |O| <= max |v|, and 1e-4 of it
            off = (o[b, :, :chunks[b]].float() - whole[b, :, at].float()).abs()
            assert not off.numel() or off.max() <= 2 * (3 * H2 + 1e-3) * v.float().abs().max()
            # scores up to 2^5, products' errors below 130 2^-24 times 2^8 on either side, the tanh's 30 2^-21
            off = (lse[b, :, :chunks[b]] - whole_lse[b, :, at]).abs()
            assert not off.numel() or off.max() <= 2 * (1e-4 + 130 * 2.0 ** -16 + 30 * 2.0 ** -21)
        done = [x + c for x, c in zip(done, chunks)]
    assert done == total


@pytest.mark.parametrize("H, Hkv, T, lens, some, window, cap, slopes, d", [
    # heads of a group that do and do not divide a row tile, groups in several units, chunks that
    # fill from none to all of the tiles that the longest one has
    (6, 2, 90, [700, 0, 300], [90, 0, 1], 0, 0.0, True, 64),
    (5, 1, 51, [130, 61], [51, 26], 0, 30.0, False, 128),
    (14, 2, 40, [0, 500, 77], [37, 2, 18], 100, 0.0, True, 128),
    (3, 1, 5, [400], None, 0, 50.0, True, 64),
    (10, 2, 3, [255, 4], [3, 1], 0, 0.0, True, 128),
    (22, 2, 2, [300, 11, 60], [1, 2, 0], 0, 20.0, True, 64),
    (7, 1, 18, [129], [17], 0, 0.0, False, 128),
    (48, 1, 9, [350, 128], [9, 4], 0, 0.0, True, 64),
    (96, 1, 3, [200], None, 0, 50.0, False, 128),
    (127, 1, 2, [100], None, 0, 0.0, True, 64),
    (131, 1, 2, [140], None, 0, 0.0, False, 64),
    (144, 1, 1, [260], None, 0, 0.0, True, 128),
    (16, 4, 700, [900, 40, 0, 1200, 3, 0], [1, 700, 0, 2, 33, 1], 0, 0.0, False, 128),
    (8, 8, 300, [0, 0], [0, 300], 0, 0.0, True, 64),
    (8, 2, 300, [50, 9], [0, 0], 0, 0.0, False, 64),
])
def test_units_of_a_group(H, Hkv, T, lens, some, window, cap, slopes, d):
    B, size = len(lens), 16
    chunks = [T] * B if some is None else some
    width = max(1, max(-(-(n + c) // size) for n, c in zip(lens, chunks)))
    table, count = tables(lens, chunks, size, width, H)
    kp, vp = pool(H, count, Hkv, size, d, "tokens"), pool(H + 1, count, Hkv, size, d, "heads")
    q = randn(H + 2, B, H, T, d)
    for b, c in enumerate(chunks):
        q[b, :, c:] = float("nan")
    sl = slopes_of(H, slopes)
    o, lse = torch.full((B, H, T, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((B, H, T), 7.0, device="cuda")
    ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(B, H, Hkv, T, width * size, d), dtype=torch.uint8, device="cuda")
    fa.fa_paged_fwd(q.cuda(), kp, vp, table.cuda(), torch.tensor(lens, **I32).cuda(),
                    None if some is None else torch.tensor(some, **I32).cuda(), o, lse, ws, 1 / math.sqrt(d), window=window,
                    cap=cap, slopes=None if sl is None else sl.cuda())
    assert fa.fa_check_device_status() == fa.FA_OK
    check_paged(q, kp, vp, table, o, lse, 1 / math.sqrt(d), lens, chunks, window, cap, sl, most=24)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dirty", [0.0, 0.2, 1.0])
def test_many_items_of_a_block(d, dirty):
    """More items of one block than a CTA keeps segments of, some of which end inside their block."""
    B, H, Hkv, T, size = 400, 16, 4, 40, 16
    g = np.random.default_rng(7)
    lens = [int(g.integers(0, 88)) if g.random() < dirty else 88 for _ in range(B)]
    table, count = tables(lens, [T] * B, size, 8, 3)
    kp, vp = pool(1, count, Hkv, size, d, "heads"), pool(2, count, Hkv, size, d, "tokens")
    for b, n in enumerate(lens):
        if (n + T) % size:
            page = int(table[b, (n + T) // size])
            kp[page, :, (n + T) % size:], vp[page, :, (n + T) % size:] = float("nan"), float("nan")
    q = randn(3, B, H, T, d).cuda()
    o, lse = torch.full_like(q, 7.0), torch.full((B, H, T), 7.0, device="cuda")
    ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(B, H, Hkv, T, 8 * size, d), dtype=torch.uint8, device="cuda")
    fa.fa_paged_fwd(q, kp, vp, table.cuda(), torch.tensor(lens, **I32).cuda(), None, o, lse, ws, 1 / math.sqrt(d))
    assert fa.fa_check_device_status() == fa.FA_OK
    assert torch.isfinite(o).all()
    check_paged(q, kp, vp, table, o, lse, 1 / math.sqrt(d), lens, [T] * B, 0, 0.0, None, most=40)


def test_offsets_past_32_bits():
    """Rows far behind 2^31 elements of a pool, of the queries and of the outputs: the bits of a pool that has
    only the pages in use, and of a request alone."""
    B, H, Hkv, T, size, d, count = 3, 4, 2, 300, 64, 128, 150000
    lens, width = [900, 0, 513], 20
    g = torch.Generator("cuda").manual_seed(1)
    need = [-(-(n + T) // size) for n in lens]
    small = [torch.randn((sum(need), Hkv, size, d), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    where = torch.arange(count - 2 * sum(need), count, 2, device="cuda")[torch.randperm(sum(need), generator=torch.Generator().manual_seed(2)).cuda()]
    big = [torch.empty((count, Hkv, size, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert int(where.min()) * Hkv * size * d > 2 ** 31
    tables_ = []
    for pages in (torch.arange(sum(need), device="cuda"), where):
        table, at = torch.full((B, width), -1, device="cuda", **I32), 0
        for b, n in enumerate(need):
            table[b, :n] = pages[at:at + n].int()
            at += n
        tables_.append(table)
    for x, y in zip(small, big):
        y[where] = x
    q = torch.randn((B, H, T, d), generator=g, device="cuda", dtype=torch.bfloat16)
    dl = torch.tensor(lens, **I32).cuda()
    one = fa.paged_attention_forward(q, *small, tables_[0], dl, 0.1)
    two = fa.paged_attention_forward(q, *big, tables_[1], dl, 0.1)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    # new rows go to the far pages too
    rows = torch.randn((B, T, H + 2 * Hkv, d), generator=g, device="cuda", dtype=torch.bfloat16)
    heads = rows[:, :, :H], rows[:, :, H:H + Hkv], rows[:, :, H + Hkv:]
    for pages, table in ((small, tables_[0]), (big, tables_[1])):
        fa.fa_rope_paged_fwd(*heads, None, None, None, None, table, dl, None, torch.empty_like(q), *pages)
    for x, y in zip(small, big):
        assert torch.equal(x, y[where])


def test_queries_past_32_bits():
    """More than 2^31 elements of queries: the last request comes out as it does alone."""
    B, H, Hkv, T, size, d = 70, 32, 4, 8000, 256, 128
    assert B * H * T * d > 2 ** 31
    g = torch.Generator("cuda").manual_seed(1)
    kp, vp = (torch.randn((40, Hkv, size, d), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.arange(32, device="cuda", **I32).repeat(B, 1)
    q = torch.randn((B, H, T, d), generator=g, device="cuda", dtype=torch.bfloat16)
    lens = torch.zeros(B, device="cuda", **I32)
    chunks = torch.full((B,), 3, device="cuda", **I32)
    chunks[-1] = T
    o, lse = fa.paged_attention_forward(q, kp, vp, table, lens, 0.1, chunks, window=600)
    # (alone an item may be cut into other parts, which rounds once more in fp32: a bf16 step of the largest)
    p, ple = fa.paged_attention_forward(q[-1:], kp, vp, table[:1], lens[:1], 0.1, window=600)
    assert float((o[-1:].float() - p.float()).abs().max()) <= 2 ** -7 * float(p.float().abs().max())
    assert float((lse[-1:] - ple).abs().max()) <= 1e-4
    assert (o[5, :, 3:] == 0).all() and (lse[5, :, 3:] == -math.inf).all()
