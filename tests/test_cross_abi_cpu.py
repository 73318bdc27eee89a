"""Refusals of the cross attention, tree and rotation entry points (no GPU): bad
arguments are turned down before anything is enqueued."""

import ctypes
import os
import struct
import subprocess

import pytest
import torch

from exact_tiled_attention_08_gb300 import fa
from exact_tiled_attention_08_gb300.build import ARCH_FLAGS, _nvcc, build_library

P = 0x7F0000000000  # aligned, never dereferenced
VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build_library()
    return fa.load_library()


def cross(lib, entry, B=1, H=4, Hkv=2, Nq=8, Nk=100, d=128, scale=0.1, ws_bytes=None, **ptr):
    size = getattr(lib, entry + "_workspace_bytes")(B, H, Hkv, Nq, Nk, d)
    names = {"fa_cross_fwd": ["q", "k", "v", "lens", "o", "lse", "ws"],
             "fa_cross_bwd": ["q", "k", "v", "lens", "o", "dout", "lse", "dq", "dk", "dv", "ws"],
             "fa_tree_fwd": ["q", "k", "v", "lens", "drafts", "masks", "o", "lse", "ws"]}[entry]
    args = [VP(ptr.get(n, P)) for n in names]
    return getattr(lib, entry)(*args, size if ws_bytes is None else ws_bytes, B, H, Hkv, Nq, Nk, d, scale, None)


@pytest.mark.parametrize("entry", ["fa_cross_fwd", "fa_cross_bwd", "fa_tree_fwd"])
def test_attention_refusals(lib, entry):
    bad = fa.FA_ERR_INVALID_ARG
    for name in ("q", "k", "v", "o", "lse", "ws"):
        assert cross(lib, entry, **{name: 0}) == bad, name
        assert cross(lib, entry, **{name: P + 4}) == fa.FA_ERR_MISALIGNED, name
    for name in ("B", "H", "Hkv", "Nq", "Nk"):
        assert cross(lib, entry, **{name: 0}) == bad and cross(lib, entry, **{name: -1}) == bad, name
    assert cross(lib, entry, H=4, Hkv=3) == bad
    assert cross(lib, entry, d=96) == fa.FA_ERR_UNSUPPORTED
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert cross(lib, entry, scale=scale) == bad
    need = getattr(lib, entry + "_workspace_bytes")(1, 4, 2, 8, 100, 128)
    assert need > 0 and cross(lib, entry, ws_bytes=need - 1) == bad
    assert cross(lib, entry, H=1 << 20, Hkv=1, Nq=1 << 11) == bad  # 2^31 rows share a head
    assert cross(lib, entry, H=1, Hkv=1, Nq=2 ** 31 - 1) == bad and cross(lib, entry, Nk=2 ** 31 - 1) == bad
    assert cross(lib, entry, B=1 << 16, H=1 << 15, Hkv=1 << 15) == bad
    assert getattr(lib, entry + "_workspace_bytes")(1, 4, 3, 8, 100, 128) == 0
    assert getattr(lib, entry + "_workspace_bytes")(1, 4, 2, 8, 100, 80) == 0


def test_argument_structs(lib):
    """The *_packed entry points check what their flat forms check; null is refused."""
    for entry, pack in fa._PACKED.items():
        assert getattr(lib, entry + "_packed")(None) == fa.FA_ERR_INVALID_ARG
    need = lib.fa_cross_fwd_workspace_bytes(1, 4, 2, 8, 100, 128)

    def call(q=P, ws_bytes=need, d=128, scale=0.1):
        return lib.fa_cross_fwd_packed(fa._PACKED["fa_cross_fwd"](q, P, P, P, P, P, P, ws_bytes, 1, 4, 2, 8, 100, d,
                                                                  scale, 0))

    assert call(q=0) == fa.FA_ERR_INVALID_ARG and call(q=P + 8) == fa.FA_ERR_MISALIGNED
    assert call(d=96) == fa.FA_ERR_UNSUPPORTED and call(scale=-1.0) == fa.FA_ERR_INVALID_ARG
    assert call(ws_bytes=need - 1) == fa.FA_ERR_INVALID_ARG
    row = (P, 1024, 1024, 128)
    args = [*row, *row, *row, P, P, P, P, P, P, P, P, 1, 2, 4, 2, 2, 128, 128, 1, 1e-6, 1.0, 0, 0]
    for at, wrong, status in ((0, P + 8, fa.FA_ERR_MISALIGNED), (25, 80, fa.FA_ERR_UNSUPPORTED),
                              (24, 1, fa.FA_ERR_INVALID_ARG), (29, float("nan"), fa.FA_ERR_INVALID_ARG)):
        bad = list(args)
        bad[at] = wrong
        assert lib.fa_rope_fwd_packed(fa._PACKED["fa_rope_fwd"](*bad)) == status, at


def test_tree_refusals(lib):
    assert cross(lib, "fa_tree_fwd", masks=P + 4) == fa.FA_ERR_MISALIGNED
    assert cross(lib, "fa_tree_fwd", lens=P + 2) == fa.FA_ERR_MISALIGNED
    assert cross(lib, "fa_tree_fwd", lens=0) == fa.FA_ERR_INVALID_ARG
    assert cross(lib, "fa_tree_fwd", Nq=65) == fa.FA_ERR_UNSUPPORTED


def test_tree_masks():
    parents = torch.tensor([[-1, 0, 0, 1, -1]])
    assert fa.tree_masks(parents).tolist() == [[1, 3, 5, 11, 16]]
    assert fa.tree_masks(torch.arange(-1, 63)[None])[0, 63] == -1  # a chain of 64 sees everything
    for wrong in ([[0]], [[-2]], [[-1, 1]]):
        with pytest.raises(ValueError):
            fa.tree_masks(torch.tensor(wrong))
    with pytest.raises(ValueError):
        fa.tree_masks(torch.full((1, 65), -1))


def rows(ptr=P, batch=1024, token=1024, head=128):
    return struct.pack("Pqqq", ptr, batch, token, head)  # fa_rows


DEFAULT = object()


def rope_fwd(lib, q=DEFAULT, k=DEFAULT, v=DEFAULT, qo=P, ko=P, vo=P, freq=P, B=1, N=2, H=4, Hkv=2, C=2, d=128, rot=128, norm=1,
             eps=1e-6, factor=1.0, inter=0, weight=P, pos=P, starts=P):
    r = [rows() if x is DEFAULT else x for x in (q, k, v)]
    return lib.fa_rope_fwd(*r, VP(weight), VP(weight), VP(freq), VP(pos), VP(starts), VP(qo), VP(ko), VP(vo), B, N, H,
                           Hkv, C, d, rot, norm, eps, factor, inter, None)


def test_rope_forward_refusals(lib):
    bad, odd, no = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_MISALIGNED, fa.FA_ERR_UNSUPPORTED
    assert rope_fwd(lib, q=None) == bad and rope_fwd(lib, qo=0) == bad and rope_fwd(lib, q=rows(ptr=0)) == bad
    assert rope_fwd(lib, q=None, k=None, v=None, qo=0, ko=0, vo=0) == bad
    for name in ("B", "N", "H", "Hkv"):
        assert rope_fwd(lib, **{name: 0}) == bad, name
    assert rope_fwd(lib, C=1) == bad and rope_fwd(lib, d=80) == no
    assert rope_fwd(lib, rot=-16) == bad and rope_fwd(lib, rot=144) == bad and rope_fwd(lib, rot=24) == no
    assert rope_fwd(lib, freq=0) == bad and rope_fwd(lib, norm=2) == bad and rope_fwd(lib, inter=-1) == bad
    assert rope_fwd(lib, eps=-1.0) == bad and rope_fwd(lib, eps=float("nan")) == bad
    assert rope_fwd(lib, factor=float("inf")) == bad
    assert rope_fwd(lib, q=rows(ptr=P + 8)) == odd and rope_fwd(lib, k=rows(token=1028)) == odd
    assert rope_fwd(lib, v=rows(head=4)) == odd and rope_fwd(lib, qo=P + 8) == odd and rope_fwd(lib, pos=P + 2) == odd
    assert rope_fwd(lib, freq=P + 4) == odd and rope_fwd(lib, weight=P + 4) == odd


def rope_bwd(lib, q=DEFAULT, k=DEFAULT, dq=DEFAULT, dk=DEFAULT, dv=DEFAULT, gq=P, gk=P, gv=P, dqw=P, dkw=P, ws=P, ws_bytes=None, N=2, H=4,
             Hkv=2, norm=1, eps=1e-6):
    r = [rows() if x is DEFAULT else x for x in (q, k, dq, dk, dv)]
    need = lib.fa_rope_bwd_workspace_bytes(1, H, Hkv, N, 128)
    return lib.fa_rope_bwd(r[0], r[1], VP(P), VP(P), VP(P), VP(P), VP(gq), VP(gk), VP(gv), r[2], r[3], r[4], VP(dqw),
                           VP(dkw), VP(ws), need if ws_bytes is None else ws_bytes, 1, N, H, Hkv, 128, 128, norm, eps,
                           1.0, 0, None)


def test_rope_backward_refusals(lib):
    bad, odd = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_MISALIGNED
    assert rope_bwd(lib, q=None) == bad and rope_bwd(lib, k=None) == bad  # the norm's gradient reads them
    assert rope_bwd(lib, dq=None) == bad and rope_bwd(lib, gv=0) == bad
    assert rope_bwd(lib, ws=0) == bad and rope_bwd(lib, ws_bytes=16) == bad
    assert rope_bwd(lib, norm=0) == bad  # weight gradients without a norm
    # gradients that overlap: a token's rows reach into the next one's, or heads share rows
    assert rope_bwd(lib, dq=rows(token=384)) == bad and rope_bwd(lib, dk=rows(head=0)) == bad
    assert rope_bwd(lib, dv=rows(head=64)) == bad
    assert rope_bwd(lib, dq=rows(ptr=P + 8)) == odd and rope_bwd(lib, ws=P + 8) == odd
    assert lib.fa_rope_bwd_workspace_bytes(1, 4, 2, 2, 100) == 0


def test_binding_refusals(lib):
    bf = dict(dtype=torch.bfloat16)
    q, kv, lse = torch.zeros((1, 4, 3, 64), **bf), torch.zeros((1, 2, 9, 64), **bf), torch.zeros((1, 4, 3))
    with pytest.raises(TypeError):
        fa.fa_cross_fwd(q.float(), kv, kv, None, q, lse, lse, 0.1, stream=0)
    with pytest.raises(ValueError):  # CPU tensors
        fa.fa_cross_fwd(q, kv, kv, None, q, lse, lse, 0.1, stream=0)
    with pytest.raises(ValueError):
        fa.fa_cross_fwd(q, kv, kv[:, :, :8], None, q, lse, lse, 0.1, stream=0)
    with pytest.raises(ValueError):
        fa.fa_rope_fwd(None, None, None, None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError):
        fa.fa_rope_fwd(q, None, None, lse, None, None, None, None, q, None, None)
    with pytest.raises(ValueError):
        fa.rope_frequencies(15)
    with pytest.raises(ValueError):
        fa.rope_frequencies(64, scaling="what")


def test_runs_of_long_items(tmp_path):
    """The backward's runs cover an item's query blocks without gaps, at the longest item too."""
    package = os.path.dirname(os.path.abspath(fa.__file__))
    source = tmp_path / "runs.cu"
    source.write_text("""
#include "fa_cross_bwd.cuh"
#include <cstdio>
int main() {
  const int blocks[] = {1, 2, 77, 607, 608, 609, 1 << 20, (1 << 24) - 2, 1 << 24};
  for (int nqb : blocks)
    for (int items = 1; items < 304; ++items) {
      const fa::CrossBwdPlan plan = fa::cross_bwd_split(items, nqb, 152);
      if (plan.parts < 1 || plan.parts > nqb || plan.rest * plan.parts > fa::kCrossBwdSlots) return 1;
      if (plan.rounds * 152 + plan.rest != items) return 2;
      for (int part = 0; part <= plan.parts; ++part)
        if (fa::cross_bwd_cut(part, plan.parts, nqb) != (long long)part * nqb / plan.parts) return 3;
    }
  return 0;
}
""")
    program = tmp_path / "runs"
    subprocess.run([_nvcc(), *ARCH_FLAGS, "-std=c++17", "-I", os.path.join(package, "csrc"), "-o", str(program),
                    str(source)], check=True, capture_output=True)
    assert subprocess.run([str(program)]).returncode == 0
