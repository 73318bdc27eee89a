"""Pages at both ends of a pool of more than 2^31 elements."""

import pytest
import torch

from exact_tiled_attention_08_gb300 import fa
from test_span_gpu import randn

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32)


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_tiled_attention_08_gb300.build import build_library

    build_library()
    fa.load_library()


@pytest.mark.parametrize("T", [1, 5, 70])
def test_pages_at_both_ends_of_a_pool(T):
    """The bits of a pool that has only the pages in use; then rotation across a border of the same pages."""
    count, Hkv, size, d = 70000, 2, 128, 128
    kp = torch.zeros((count, Hkv, size, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    assert kp.numel() > 2 ** 31
    kk, vv = randn(1, 4, Hkv, size, d).cuda(), randn(2, 4, Hkv, size, d).cuda()
    table = torch.tensor([[0, count - 1, 66000, 3]], **I32).cuda()
    for i, page in enumerate(table[0].tolist()):
        kp[page], vp[page] = kk[i], vv[i]
    q = randn(3, 1, 4, T, d).cuda()
    lens = torch.tensor([512 - T], **I32).cuda()
    far = fa.paged_attention_forward(q, kp, vp, table, lens, 0.1)
    near = fa.paged_attention_forward(q, kk, vv, torch.arange(4, **I32)[None].cuda(), lens, 0.1)
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
    rows = randn(4, 1, T, Hkv, d).cuda()
    at = 256 - (T + 1) // 2
    fa.fa_rope_paged_fwd(None, rows, rows, None, None, None, None, table, torch.tensor([at], **I32).cuda(), None, None,
                         kp, vp)
    for pages, was in ((kp, kk), (vp, vv)):
        want = was[1:3].transpose(1, 2).reshape(2 * size, Hkv, d).clone()
        want[at - size:at - size + T] = rows[0]
        got = pages[[count - 1, 66000]].transpose(1, 2).reshape(2 * size, Hkv, d)
        assert torch.equal(got, want)
        assert torch.equal(pages[0], was[0]) and torch.equal(pages[3], was[3])
