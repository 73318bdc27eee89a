"""Refusals of the span attention, paged attention and paged rotation entry points (no
GPU): bad arguments are turned down before anything is enqueued."""

import ctypes
import struct

import pytest
import torch

from exact_tiled_attention_08_gb300 import fa
from exact_tiled_attention_08_gb300.build import build_library

P = 0x7F0000000000  # aligned, never dereferenced
VP = ctypes.c_void_p
BAD, ODD, NO = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_MISALIGNED, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_library()
    return fa.load_library()


def span(lib, entry, B=1, H=4, Hkv=2, N=100, d=128, scale=0.1, cap=0.0, window=0, causal=1, ws_bytes=None, **ptr):
    need = getattr(lib, entry + "_workspace_bytes")(B, H, Hkv, N, d)
    names = {"fa_span_fwd": ["q", "k", "v", "begin", "end", "slopes", "o", "lse", "ws"],
             "fa_span_bwd": ["q", "k", "v", "begin", "end", "slopes", "o", "dout", "lse", "dq", "dk", "dv", "ws"]}[entry]
    return getattr(lib, entry)(*(VP(ptr.get(n, P)) for n in names), need if ws_bytes is None else ws_bytes, B, H, Hkv,
                               N, d, scale, cap, window, causal, None)


@pytest.mark.parametrize("entry", ["fa_span_fwd", "fa_span_bwd"])
def test_span_refusals(lib, entry):
    pointers = ["q", "k", "v", "o", "lse", "ws"] + (["dout", "dq", "dk", "dv"] if entry == "fa_span_bwd" else [])
    for name in pointers:
        assert span(lib, entry, **{name: 0}) == BAD and span(lib, entry, **{name: P + 4}) == ODD, name
    for name in ("begin", "end", "slopes"):
        assert span(lib, entry, **{name: P + 2}) == ODD, name
    for name in ("B", "H", "Hkv", "N"):
        assert span(lib, entry, **{name: 0}) == BAD and span(lib, entry, **{name: -1}) == BAD, name
    assert span(lib, entry, H=4, Hkv=3) == BAD and span(lib, entry, d=96) == NO
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert span(lib, entry, scale=scale) == BAD
    for cap in (-1.0, float("nan"), float("inf"), 1e-42):  # (the last: scale / cap is infinite)
        assert span(lib, entry, cap=cap) == BAD, cap
    assert span(lib, entry, window=-1) == BAD and span(lib, entry, causal=2) == BAD and span(lib, entry, causal=-1) == BAD
    need = getattr(lib, entry + "_workspace_bytes")(1, 4, 2, 100, 128)
    assert need > 0 and span(lib, entry, ws_bytes=need - 1) == BAD
    assert span(lib, entry, N=2 ** 31 - 1) == BAD and span(lib, entry, B=1 << 16, H=1 << 15, Hkv=1 << 15) == BAD
    assert getattr(lib, entry + "_workspace_bytes")(1, 4, 3, 100, 128) == 0
    assert getattr(lib, entry + "_workspace_bytes")(1, 4, 2, 100, 80) == 0
    # addresses that no allocation covers (or, without a GPU, no device to ask)
    assert span(lib, entry) in (BAD, fa.FA_ERR_CUDA)


def pages(ptr=P, page=4096, head=2048, token=128):
    return struct.pack("Pqqq", ptr, page, head, token)  # fa_pages


def paged(lib, kp=None, vp=None, B=1, H=4, Hkv=2, T=3, d=128, count=5, size=16, width=4, scale=0.1, cap=0.0, window=0,
          ws_bytes=None, **ptr):
    need = lib.fa_paged_fwd_workspace_bytes(B, H, Hkv, T, max(1, min(width * size, 2 ** 31 - 1)), d)
    p = [VP(ptr.get(n, P)) for n in ("q", "table", "lens", "chunks", "slopes", "o", "lse", "ws")]
    return lib.fa_paged_fwd(p[0], pages() if kp is None else kp, pages() if vp is None else vp, *p[1:],
                            need if ws_bytes is None else ws_bytes, B, H, Hkv, T, d, count, size, width, scale, cap,
                            window, None)


def test_paged_refusals(lib):
    for name in ("q", "o", "lse", "ws"):
        assert paged(lib, **{name: 0}) == BAD and paged(lib, **{name: P + 4}) == ODD, name
    for name in ("table", "lens"):
        assert paged(lib, **{name: 0}) == BAD and paged(lib, **{name: P + 2}) == ODD, name
    assert paged(lib, chunks=P + 2) == ODD and paged(lib, slopes=P + 2) == ODD
    for name in ("B", "H", "Hkv", "T", "count", "size", "width"):
        assert paged(lib, **{name: 0}) == BAD and paged(lib, **{name: -1}) == BAD, name
    for size in (1, 8, 24, 48, 100):
        assert paged(lib, size=size) == NO, size
    for which in ("kp", "vp"):
        assert paged(lib, **{which: pages(ptr=0)}) == BAD and paged(lib, **{which: pages(ptr=P + 8)}) == ODD
        for stride in ("page", "head", "token"):
            assert paged(lib, **{which: pages(**{stride: 0})}) == BAD, stride
            assert paged(lib, **{which: pages(**{stride: -128})}) == BAD, stride
            assert paged(lib, **{which: pages(**{stride: 132})}) == ODD, stride
            assert paged(lib, **{which: pages(**{stride: 1 << 38})}) == BAD, stride
    assert lib.fa_paged_fwd(VP(P), None, pages(), *[VP(P)] * 7, 1 << 30, 1, 4, 2, 3, 128, 5, 16, 4, 0.1, 0.0, 0, None) == BAD
    assert paged(lib, d=96) == NO and paged(lib, H=4, Hkv=3) == BAD
    assert paged(lib, scale=0.0) == BAD and paged(lib, cap=-2.0) == BAD and paged(lib, window=-1) == BAD
    assert paged(lib, width=1 << 27, size=16) == BAD  # 2^31 tokens
    need = lib.fa_paged_fwd_workspace_bytes(1, 4, 2, 3, 64, 128)
    assert need > 0 and paged(lib, ws_bytes=need - 1) == BAD
    assert paged(lib) in (BAD, fa.FA_ERR_CUDA)


def rows(ptr=P, batch=1024, token=1024, head=128):
    return struct.pack("Pqqq", ptr, batch, token, head)  # fa_rows


DEFAULT = object()


def rope(lib, q=DEFAULT, k=DEFAULT, v=DEFAULT, kp=DEFAULT, vp=DEFAULT, qo=P, B=1, N=2, H=4, Hkv=2, d=128, count=5,
         size=16, width=4, rot=128, norm=1, eps=1e-6, factor=1.0, inter=0, **ptr):
    r = [rows() if x is DEFAULT else x for x in (q, k, v)]
    g = [pages() if x is DEFAULT else x for x in (kp, vp)]
    p = [VP(ptr.get(n, P)) for n in ("qw", "kw", "freq", "pos", "table", "lens", "chunks")]
    return lib.fa_rope_paged_fwd(*r, *p, VP(qo), *g, B, N, H, Hkv, d, count, size, width, rot, norm, eps, factor, inter,
                                 None)


def test_rope_paged_refusals(lib):
    assert rope(lib, q=None) == BAD and rope(lib, qo=0) == BAD and rope(lib, k=None) == BAD and rope(lib, kp=None) == BAD
    assert rope(lib, vp=pages(ptr=0)) == BAD and rope(lib, v=rows(ptr=0)) == BAD
    assert rope(lib, q=None, k=None, v=None, kp=None, vp=None, qo=0) == BAD
    for name in ("B", "N", "H", "Hkv", "count", "size", "width"):
        assert rope(lib, **{name: 0}) == BAD, name
    assert rope(lib, table=0) == BAD and rope(lib, lens=0) == BAD
    for name in ("table", "lens", "chunks", "pos"):
        assert rope(lib, **{name: P + 2}) == ODD, name
    for size in (8, 48):
        assert rope(lib, size=size) == NO
    assert rope(lib, kp=pages(ptr=P + 8)) == ODD and rope(lib, vp=pages(token=132)) == ODD
    # rows that share memory: pages, heads or tokens closer than they are long
    assert rope(lib, kp=pages(page=2048)) == BAD and rope(lib, vp=pages(head=1024)) == BAD
    assert rope(lib, kp=pages(token=64)) == BAD and rope(lib, kp=pages(token=256, head=128)) in (BAD, fa.FA_ERR_CUDA)
    assert rope(lib, d=80) == NO and rope(lib, rot=24) == NO and rope(lib, rot=144) == BAD
    assert rope(lib, eps=-1.0) == BAD and rope(lib, factor=float("nan")) == BAD and rope(lib, norm=2) == BAD
    assert rope(lib, q=rows(ptr=P + 8)) == ODD and rope(lib, k=rows(token=1028)) == ODD
    assert rope(lib) in (BAD, fa.FA_ERR_CUDA)


def test_argument_structs_hold_what_the_flat_forms_take(lib):
    """One wrong argument at a time, through the structs."""
    need = lib.fa_span_fwd_workspace_bytes(1, 4, 2, 100, 128)
    args = [P] * 9 + [need, 1, 4, 2, 100, 128, 0.1, 0.0, 0, 1, 0]
    for at, wrong, status in ((3, P + 2, ODD), (5, P + 2, ODD), (8, 0, BAD), (9, need - 1, BAD), (13, 0, BAD), (14, 96, NO),
                              (15, -1.0, BAD), (16, -1.0, BAD), (17, -1, BAD), (18, 2, BAD)):
        bad = list(args)
        bad[at] = wrong
        assert lib.fa_span_fwd_packed(fa._PACKED["fa_span_fwd"](*bad)) == status, at
    need = lib.fa_span_bwd_workspace_bytes(1, 4, 2, 100, 128)
    args = [P] * 13 + [need, 1, 4, 2, 100, 128, 0.1, 0.0, 0, 1, 0]
    for at, wrong, status in ((4, P + 2, ODD), (7, 0, BAD), (13, need - 1, BAD), (18, 96, NO), (20, -1.0, BAD), (22, 2, BAD)):
        bad = list(args)
        bad[at] = wrong
        assert lib.fa_span_bwd_packed(fa._PACKED["fa_span_bwd"](*bad)) == status, at
    page = (P, 4096, 2048, 128)
    need = lib.fa_paged_fwd_workspace_bytes(1, 4, 2, 3, 64, 128)
    args = [P, *page, *page, *[P] * 7, need, 1, 4, 2, 3, 128, 5, 16, 4, 0.1, 0.0, 0, 0]
    for at, wrong, status in ((4, 132, ODD), (8, 0, BAD), (10, P + 2, ODD), (16, need - 1, BAD), (21, 96, NO), (23, 24, NO),
                              (24, 0, BAD), (26, -1.0, BAD), (27, -1, BAD)):
        bad = list(args)
        bad[at] = wrong
        assert lib.fa_paged_fwd_packed(fa._PACKED["fa_paged_fwd"](*bad)) == status, at
    row = (P, 1024, 1024, 128)
    args = [*row, *row, *row, *[P] * 8, *page, *page, 1, 2, 4, 2, 128, 5, 16, 4, 128, 1, 1e-6, 1.0, 0, 0]
    for at, wrong, status in ((0, P + 8, ODD), (17, P + 2, ODD), (20, P + 8, ODD), (21, 2048, BAD), (32, 80, NO),
                              (34, 24, NO), (36, 24, NO), (38, -1.0, BAD), (40, 2, BAD)):
        bad = list(args)
        bad[at] = wrong
        assert lib.fa_rope_paged_fwd_packed(fa._PACKED["fa_rope_paged_fwd"](*bad)) == status, at


def test_binding_refusals(lib):
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    q, kv, lse = torch.zeros((1, 4, 9, 64), **bf), torch.zeros((1, 2, 9, 64), **bf), torch.zeros((1, 4, 9))
    for wrong in (dict(q=q.float()), dict(k=kv[:, :, :8]), dict(begin=torch.zeros((1, 9))), dict(lse=lse.double())):
        x = dict(q=q, k=kv, v=kv, begin=None, end=None, o=q, lse=lse) | wrong
        with pytest.raises((TypeError, ValueError)):
            fa.fa_span_fwd(*x.values(), lse, 0.1, stream=0)
    with pytest.raises(ValueError):  # CPU tensors
        fa.fa_span_fwd(q, kv, kv, None, None, q, lse, lse, 0.1, stream=0)
    kp, table, lens = torch.zeros((3, 2, 16, 64), **bf), torch.zeros((1, 2), **i32), torch.zeros((1,), **i32)
    for wrong in (dict(kp=kp.transpose(2, 3)), dict(vp=kp[:2]), dict(table=table[0]), dict(table=table.long()),
                  dict(lens=lens.long()), dict(kp=kp.float())):
        x = dict(q=q, kp=kp, vp=kp, table=table, lens=lens, chunks=None, o=q, lse=lse) | wrong
        with pytest.raises((TypeError, ValueError)):
            fa.fa_paged_fwd(*x.values(), lse, 0.1, stream=0)
    with pytest.raises(ValueError):
        fa.fa_rope_paged_fwd(None, None, None, None, None, None, None, table, lens, None, None, kp, kp)
    with pytest.raises(ValueError):
        fa.fa_rope_paged_fwd(q, None, None, lse, None, None, None, None, None, None, q, None, None)
