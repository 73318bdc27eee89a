"""The cross attention, cache and rotation entry points as they are used together,
and the calls around their edges: other alignments, streams at the same time,
many requests, waits that run out."""

import math

import numpy as np
import pytest
import torch

from exact_tiled_attention_08_gb300 import fa
from oracle.cross import masked_attention_ref, rope_ref

pytestmark = pytest.mark.gpu

H2 = 2.0 ** -8  # half a step of bf16, relative


@pytest.fixture(autouse=True)
def built():
    from exact_tiled_attention_08_gb300.build import build_library

    build_library()
    fa.load_library()
    yield
    fa.fa_debug_stall(False)
    fa.fa_set_wait_limit_ns(0)


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def workspace(nbytes):
    return torch.empty(max(16, nbytes), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("d", [64, 128])
def test_serving_steps(d):
    """Prompt, then single tokens, then a drafted tree of which a path is kept: each
    step rotates and appends to the cache and attends to it.  The last tokens'
    outputs against one attention in fp64 over all the tokens kept.

    Bound: K and V of the cache are bf16 roundings of the oracle's own K; a score
    is off by at most 2 H |q||k| scale (both sides rounded) from the oracle's, so P
    by twice that relatively, plus test_cross_gpu's bounds."""
    B, H, Hkv, C, eps, scale = 2, 4, 2, 400, 1e-6, 1 / math.sqrt(d)
    freq, factor = fa.rope_frequencies(d, scaling="parts", scale=4.0, trained_len=128)
    wq, wk = (torch.rand(d, generator=torch.Generator().manual_seed(s)).cuda() + 0.5 for s in (1, 2))
    kc, vc = (torch.full((B, Hkv, C, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    kept = [[] for _ in range(B)]  # projection rows [H + 2 Hkv, d] of the tokens kept

    def step(rows, positions, masks=None):
        T = rows.shape[1]
        q = torch.empty((B, H, T, d), dtype=torch.bfloat16, device="cuda")
        fa.fa_rope_fwd(rows[:, :, :H], rows[:, :, H:H + Hkv], rows[:, :, H + Hkv:], wq, wk, freq, positions, lens, q, kc,
                       vc, eps=eps, factor=factor)
        return fa.tree_attention_forward(q, kc, vc, lens, scale, draft_masks=masks)

    seed = 10
    for T in (150, 1, 1):
        rows = randn(seed, B, T, H + 2 * Hkv, d)
        seed += 1
        o, lse = step(rows, None)
        for b in range(B):
            kept[b] += list(host(rows[b]))
        lens += T
    parents = torch.tensor([[-1, 0, 0, 2, 2], [-1, -1, 1, 2, 0]])
    depth = torch.tensor([[0, 1, 1, 2, 2], [0, 0, 1, 2, 1]], dtype=torch.int32).cuda()
    rows = randn(seed, B, 5, H + 2 * Hkv, d)
    o, lse = step(rows, lens[:, None] + depth, fa.tree_masks(parents).cuda())
    paths = [[0, 2, 4], [1, 2, 3]]  # to the draft whose output is checked
    for b, path in enumerate(paths):
        tokens = np.stack(kept[b] + [host(rows[b, t]) for t in path])
        pos = np.arange(len(tokens))
        args = freq.cpu().numpy(), pos, eps, factor
        q = rope_ref(tokens[:, :H].transpose(1, 0, 2), wq.cpu().numpy(), *args)
        k = rope_ref(tokens[:, H:H + Hkv].transpose(1, 0, 2), wk.cpu().numpy(), *args)
        v = tokens[:, H + Hkv:].transpose(1, 0, 2)
        for h in range(H):
            j = h // (H // Hkv)
            ro, rl, size = masked_attention_ref(q[h, -1:], k[j], v[j], scale, np.ones((1, len(tokens)), bool))
            off = 2 * H2 * np.linalg.norm(q[h, -1]) * np.linalg.norm(k[j], axis=1).max() * scale
            err = np.abs(host(o[b, h, path[-1]]) - ro[0])
            assert (err <= 2 * off * size[0] + H2 * (size[0] + 2 * np.abs(ro[0])) + 1e-4).all(), (b, h, err.max(), off)
            assert abs(float(lse[b, h, path[-1]]) - rl[0]) <= off + 1e-4


def grad_error(got, want):
    want = want.detach()
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("d", [64, 128])
def test_training_layer(d):
    """Self-attention (norm and rotation, causal) and cross attention (norm only) of one
    decoder layer, forward and backward, against autograd in fp64.

    Between input and gradient each path rounds at most eight times to bf16 (q or k,
    P, O, dP's operands, dS, dq or dk, the gradient): in the 2-norm 8 H in the worst
    case, the bound taken."""
    B, N, M, H, eps, scale = 2, 190, 140, 2, 1e-5, 1 / math.sqrt(d)
    lens = [140, 75]
    x, y = randn(1, B, N, 4 * H, d), randn(2, B, M, 2 * H, d)  # q, k, v and cross q; cross k, v
    w = [torch.rand(d, generator=torch.Generator().manual_seed(s)).cuda() + 0.5 for s in range(3, 7)]
    do1, do2 = randn(8, B, H, N, d), randn(9, B, H, N, d)
    freq, _ = fa.rope_frequencies(d)
    kl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    head = lambda n: torch.empty((B, H, n, d), dtype=torch.bfloat16, device="cuda")
    q, k, v, cq, ck, cv = head(N), head(N), head(N), head(N), head(M), head(M)
    xs = [x[:, :, i * H:(i + 1) * H] for i in range(4)]
    ys = [y[:, :, i * H:(i + 1) * H] for i in range(2)]
    fa.fa_rope_fwd(xs[0], xs[1], xs[2], w[0], w[1], freq, None, None, q, k, v, eps=eps)
    fa.fa_rope_fwd(xs[3], None, None, w[2], None, None, None, None, cq, None, None, eps=eps)
    fa.fa_rope_fwd(None, ys[0], ys[1], None, w[3], None, None, None, None, ck, cv, eps=eps)
    o1, l1 = fa.attention_forward(q, k, v, scale, True)
    o2, l2 = fa.cross_attention_forward(cq, ck, cv, scale, kl)
    dq, dk, dv = fa.attention_backward(q, k, v, o1, do1, l1, scale, True)
    dcq, dck, dcv = fa.cross_attention_backward(cq, ck, cv, o2, do2, l2, scale, kl)
    dx, dy = torch.empty_like(x), torch.empty_like(y)
    dxs = [dx[:, :, i * H:(i + 1) * H] for i in range(4)]
    dys = [dy[:, :, i * H:(i + 1) * H] for i in range(2)]
    dw = [torch.empty(d, device="cuda") for _ in range(4)]
    ws = workspace(fa.fa_rope_bwd_workspace_bytes(B, H, H, N, d))
    fa.fa_rope_bwd(xs[0], xs[1], w[0], w[1], freq, None, dq, dk, dv, dxs[0], dxs[1], dxs[2], dw[0], dw[1], ws, eps=eps)
    fa.fa_rope_bwd(xs[3], None, w[2], None, None, None, dcq, None, None, dxs[3], None, None, dw[2], None, ws, eps=eps)
    fa.fa_rope_bwd(None, ys[0], None, w[3], None, None, None, dck, dcv, None, dys[0], dys[1], None, dw[3], ws, eps=eps)

    X, Y = x.double().requires_grad_(), y.double().requires_grad_()
    W = [t.double().requires_grad_() for t in w]

    def norm(t, wt):
        return (t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps) * wt).transpose(1, 2)

    def turn(t):
        a = torch.arange(N, device="cuda", dtype=torch.float64)[:, None] * freq
        lo, hi = t[..., :d // 2], t[..., d // 2:]
        return torch.cat((lo * a.cos() - hi * a.sin(), lo * a.sin() + hi * a.cos()), -1)

    s = scale * turn(norm(X[:, :, :H], W[0])) @ turn(norm(X[:, :, H:2 * H], W[1])).transpose(-1, -2)
    s = s.masked_fill(torch.ones(N, N, device="cuda").triu(1).bool(), -math.inf)
    r1 = torch.softmax(s, -1) @ X[:, :, 2 * H:3 * H].transpose(1, 2)
    s = scale * norm(X[:, :, 3 * H:], W[2]) @ norm(Y[:, :, :H], W[3]).transpose(-1, -2)
    s = s.masked_fill(torch.arange(M, device="cuda") >= kl[:, None, None, None], -math.inf)
    r2 = torch.softmax(s, -1) @ Y[:, :, H:].transpose(1, 2)
    ((r1 * do1).sum() + (r2 * do2).sum()).backward()
    assert grad_error(o1, r1) <= 8 * H2 and grad_error(o2, r2) <= 8 * H2
    for i in range(4):
        assert grad_error(dxs[i], X.grad[:, :, i * H:(i + 1) * H]) <= 8 * H2, i
    for i in range(2):
        assert grad_error(dys[i], Y.grad[:, :, i * H:(i + 1) * H]) <= 8 * H2, i
    for i in range(4):
        assert grad_error(dw[i], W[i].grad) <= 8 * H2, i
    assert (dy[1, lens[1]:] == 0).all()


def shifted(t, elements=8):
    """t at an address 16 bytes past a 32-byte boundary."""
    raw = torch.empty(t.numel() + 32, dtype=t.dtype, device=t.device)
    out = raw[elements:elements + t.numel()].view(t.shape)
    assert out.data_ptr() % 32 == 16
    return out.copy_(t)


def test_addresses_on_16_byte_boundaries():
    B, H, Hkv, Nq, Nk, d = 2, 4, 2, 150, 300, 128
    q, k, v, do = randn(1, B, H, Nq, d), randn(2, B, Hkv, Nk, d), randn(3, B, Hkv, Nk, d), randn(4, B, H, Nq, d)
    o, lse = fa.cross_attention_forward(q, k, v, 0.1)
    dq, dk, dv = fa.cross_attention_backward(q, k, v, o, do, lse, 0.1)
    q2, k2, v2, do2, o2 = (shifted(t) for t in (q, k, v, do, torch.zeros_like(o)))
    lse2 = shifted(torch.zeros_like(lse), 4)
    g2 = [shifted(torch.zeros_like(t)) for t in (dq, dk, dv)]
    wf = workspace(fa.fa_cross_fwd_workspace_bytes(B, H, Hkv, Nq, Nk, d) + 16)[16:]
    wb = workspace(fa.fa_cross_bwd_workspace_bytes(B, H, Hkv, Nq, Nk, d) + 16)[16:]
    assert wf.data_ptr() % 256 == 16
    fa.fa_cross_fwd(q2, k2, v2, None, o2, lse2, wf, 0.1)
    fa.fa_cross_bwd(q2, k2, v2, None, o2, do2, lse2, *g2, wb, 0.1)
    assert fa.fa_check_device_status() == fa.FA_OK
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(dk, g2[1]) and torch.equal(dv, g2[2])
    assert torch.allclose(dq.float(), g2[0].float(), rtol=2 * H2, atol=1e-5)
    # one key block: dQ is written directly
    k3, v3 = k[:, :, :100].contiguous(), v[:, :, :100].contiguous()
    want = fa.cross_attention_backward(q, k3, v3, o, do, lse, 0.1)
    g3 = [shifted(torch.zeros_like(t)) for t in want]
    fa.fa_cross_bwd(q2, k3, v3, None, o2, do2, lse2, *g3, wb, 0.1)
    for a, b in zip(want, g3):
        assert torch.equal(a, b)


def test_calls_on_two_streams_at_once():
    """Each stream with outputs and workspace of its own; results as alone."""
    B, H, Hkv, Nq, Nk, d = 2, 8, 4, 70, 1500, 128
    sets = []
    for s in range(2):
        q, k, v, do = (randn(10 * s + i, *sh) for i, sh in enumerate([(B, H, Nq, d), (B, Hkv, Nk, d), (B, Hkv, Nk, d),
                                                                      (B, H, Nq, d)]))
        o, lse = fa.cross_attention_forward(q, k, v, 0.09)
        grads = fa.cross_attention_backward(q, k, v, o, do, lse, 0.09)
        sets.append((q, k, v, do, o, lse, grads))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    outs = []
    for st, (q, k, v, do, o, lse, grads) in zip(streams, sets):
        with torch.cuda.stream(st):
            outs.append((torch.empty_like(o), torch.empty_like(lse), [torch.empty_like(g) for g in grads],
                         workspace(fa.fa_cross_fwd_workspace_bytes(B, H, Hkv, Nq, Nk, d)),
                         workspace(fa.fa_cross_bwd_workspace_bytes(B, H, Hkv, Nq, Nk, d))))
    torch.cuda.synchronize()
    for _ in range(4):
        for st, (q, k, v, do, o, lse, grads), (o2, l2, g2, wf, wb) in zip(streams, sets, outs):
            fa.fa_cross_fwd(q, k, v, None, o2, l2, wf, 0.09, stream=st)
            fa.fa_cross_bwd(q, k, v, None, o2, do, l2, *g2, wb, 0.09, stream=st)
    torch.cuda.synchronize()
    assert fa.fa_check_device_status() == fa.FA_OK
    for (q, k, v, do, o, lse, grads), (o2, l2, g2, wf, wb) in zip(sets, outs):
        assert torch.equal(o, o2) and torch.equal(lse, l2)
        assert torch.equal(grads[1], g2[1]) and torch.equal(grads[2], g2[2])


@pytest.mark.parametrize("d", [64, 128])
def test_many_requests_of_any_length(d):
    """More requests than a warp has lanes, lengths of zero among them; each request
    alone gives the same rows (its key blocks are cut elsewhere: within the bounds of
    two results)."""
    B, H, Hkv, C, T = 150, 4, 2, 700, 3
    q, k, v = randn(1, B, H, T, d), randn(2, B, Hkv, C, d), randn(3, B, Hkv, C, d)
    g = torch.Generator().manual_seed(4)
    lens = (torch.rand(B, generator=g) ** 3 * (C - T)).to(torch.int32)
    lens[::17] = 0
    o, lse = fa.tree_attention_forward(q, k, v, lens.cuda(), 0.11)
    kl = lens.clone().cuda()
    co, cl = fa.cross_attention_forward(q, k, v, 0.11, kl)
    do = randn(5, B, H, T, d)
    cg = fa.cross_attention_backward(q, k, v, co, do, cl, 0.11, kl)
    for b in (0, 1, 17, 33, 80, 149):
        one = slice(b, b + 1)
        args = [t[one].contiguous() for t in (q, k, v)]
        oo, ll = fa.tree_attention_forward(*args, lens[one].cuda(), 0.11)
        size = v[b].float().abs().max()
        assert (oo[0].float() - o[b].float()).abs().max() <= 4 * H2 * size
        assert torch.allclose(ll[0], lse[b], atol=2e-4)
        oo, ll = fa.cross_attention_forward(*args, 0.11, kl[one])
        assert (oo[0].float() - co[b].float()).abs().max() <= 4 * H2 * size
        assert torch.equal(ll[0] == -math.inf, cl[b] == -math.inf)
        gg = fa.cross_attention_backward(*args, co[one].contiguous(), do[one].contiguous(), cl[one].contiguous(), 0.11,
                                         kl[one])
        for a, w in zip(gg, cg):
            assert torch.allclose(a[0].float(), w[b].float(), rtol=2 * H2, atol=1e-4), b
        assert (cg[1][b, :, int(lens[b]):] == 0).all()


def test_waits_that_run_out_are_reported():
    B, H, Hkv, Nq, Nk, d = 1, 4, 2, 40, 900, 128
    q, k, v, do = randn(1, B, H, Nq, d), randn(2, B, Hkv, Nk, d), randn(3, B, Hkv, Nk, d), randn(4, B, H, Nq, d)
    lens = torch.tensor([850], dtype=torch.int32, device="cuda")
    o, lse = fa.cross_attention_forward(q, k, v, 0.1, lens)
    dq, dk, dv = fa.cross_attention_backward(q, k, v, o, do, lse, 0.1, lens)
    fa.fa_set_wait_limit_ns(1_000_000)
    fa.fa_debug_stall(True)
    for call in (lambda: fa.cross_attention_forward(q, k, v, 0.1, lens),
                 lambda: fa.cross_attention_backward(q, k, v, o, do, lse, 0.1, lens),
                 lambda: fa.tree_attention_forward(q, k, v, lens, 0.1)):
        with pytest.raises(fa.FaError) as err:
            call()
        assert err.value.status == fa.FA_ERR_TIMEOUT
    fa.fa_debug_stall(False)
    fa.fa_set_wait_limit_ns(0)
    o2, lse2 = fa.cross_attention_forward(q, k, v, 0.1, lens)
    g = fa.cross_attention_backward(q, k, v, o2, do, lse2, 0.1, lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(dk, g[1]) and torch.equal(dv, g[2])


def test_refusals_on_the_device():
    q, kv = randn(1, 1, 4, 3, 64), randn(2, 1, 2, 9, 64)
    o, lse = torch.empty_like(q), torch.empty((1, 4, 3), device="cuda")
    ws = workspace(fa.fa_cross_fwd_workspace_bytes(1, 4, 2, 3, 9, 64))
    lens = torch.tensor([9], dtype=torch.int32, device="cuda")
    bad = [
        lambda: fa.fa_cross_fwd(q, kv, kv, lens.long(), o, lse, ws, 0.1),           # lengths of another type
        lambda: fa.fa_cross_fwd(q, kv, kv, lens.cpu(), o, lse, ws, 0.1),            # on the host
        lambda: fa.fa_cross_fwd(q, kv, kv.transpose(1, 2), None, o, lse, ws, 0.1),  # not contiguous
        lambda: fa.fa_cross_fwd(q[:, :3].contiguous(), kv, kv, None, o[:, :3].contiguous(), lse[:, :3].contiguous(), ws,
                                0.1),                                               # 3 heads over 2
        lambda: fa.fa_cross_fwd(q, kv, kv, None, o, lse, ws[:16], 0.1),             # small workspace
        lambda: fa.fa_cross_fwd(q, kv, kv, None, o, lse, ws, 0.0),
        lambda: fa.fa_tree_fwd(q, kv, kv, None, None, None, o, lse, ws, 0.1),       # no lengths
        lambda: fa.fa_rope_fwd(q.transpose(1, 2)[..., ::2], None, None, None, None, None, None, None, o, None, None),
        lambda: fa.fa_rope_fwd(q.transpose(1, 2), None, None, None, None, fa.rope_frequencies(24)[0], None, None, o, None,
                               None),                                               # 24 is not a multiple of 16
    ]
    for call in bad:
        with pytest.raises((TypeError, ValueError, AttributeError, fa.FaError)):
            call()
    host_lens = torch.tensor([9], dtype=torch.int32)
    st = fa.load_library().fa_cross_fwd(q.data_ptr(), kv.data_ptr(), kv.data_ptr(), host_lens.data_ptr(),
                                        o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), 1, 4, 2, 3, 9, 64, 0.1,
                                        0)
    assert st == fa.FA_ERR_INVALID_ARG  # host memory, refused before anything runs
    assert fa.fa_check_device_status() == fa.FA_OK
