"""The conveniences of the binding called with a stream that is not the current
one: what they allocate and fill is ordered with the call, and neither stream is
given memory that the other still works on."""

import pytest
import torch

from exact_tiled_attention_08_gb300 import fa

pytestmark = pytest.mark.gpu

B, H, N, d = 2, 4, 200, 128
BUSY = 40_000_000  # cycles: some 20 ms


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_tiled_attention_08_gb300.build import build_library

    build_library()
    fa.load_library()
    assert torch.cuda.is_available()


def calls():
    g = torch.Generator("cuda").manual_seed(3)
    q, k, v, do = (torch.randn((B, H, N, d), generator=g, device="cuda").bfloat16() for _ in range(4))
    signs = torch.where(torch.rand((d,), generator=g, device="cuda") < 0.5, 1, -1).to(torch.int8)
    lens = torch.tensor([N, 50], dtype=torch.int32, device="cuda")
    behind = torch.tensor([N - 9, 50], dtype=torch.int32, device="cuda")
    drafts = torch.tensor([9, 4], dtype=torch.int32, device="cuda")
    new = q[:, :, :9].contiguous()
    o, lse = fa.attention_forward(q, k, v, 0.1)
    oc, lc = fa.cross_attention_forward(q, k, v, 0.1, lens)
    return {  # entry point, and a call of the convenience
        "attention_forward": ("fa_fwd", lambda **kw: fa.attention_forward(q, k, v, 0.1, **kw)),
        "attention_forward_fp8": ("fa_fwd_fp8", lambda **kw: fa.attention_forward_fp8(q, k, v, signs, 0.1, **kw)),
        "attention_backward": ("fa_bwd_deterministic", lambda **kw: fa.attention_backward(q, k, v, o, do, lse, 0.1,
                                                                                         deterministic=True, **kw)),
        "cross_attention_forward": ("fa_cross_fwd", lambda **kw: fa.cross_attention_forward(q, k, v, 0.1, lens, **kw)),
        "cross_attention_backward": ("fa_cross_bwd", lambda **kw: fa.cross_attention_backward(q, k, v, oc, do, lc, 0.1, lens,
                                                                                              **kw)[1:]),
        "tree_attention_forward": ("fa_tree_fwd", lambda **kw: fa.tree_attention_forward(new, k, v, behind, 0.1, drafts, **kw)),
    }


NAMES = ["attention_forward", "attention_forward_fp8", "attention_backward", "cross_attention_forward",
         "cross_attention_backward", "tree_attention_forward"]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_call_on_another_stream_than_the_current_one(name, raw):
    """The current stream is busy: a fill that waited there would land behind the result."""
    call = calls()[name][1]
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    got = call(stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_default_stream_by_its_handle():
    call = calls()["tree_attention_forward"][1]
    want, got = call(), call(stream=0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("name", NAMES[1:])
def test_workspace_is_not_given_to_the_current_stream(name, monkeypatch):
    """A call left running on a side stream: its workspace is freed for that stream only."""
    entry, call = calls()[name]
    real, seen = getattr(fa, entry), []

    def spy(*args, **kw):
        seen.extend((t.data_ptr(), t.numel()) for t in args if isinstance(t, torch.Tensor) and t.dtype == torch.uint8)
        return real(*args, **kw)

    monkeypatch.setattr(fa, entry, spy)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = call(stream=side, check_status=False)
    (address, size), = seen
    again = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() != address
    torch.cuda.synchronize()
    assert fa.fa_check_device_status() == fa.FA_OK and not any(t.isnan().any() for t in got)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_not_given_back_while_the_current_stream_reads_them(name):
    call = calls()[name][1]
    side = torch.cuda.Stream()
    got = call(stream=side)
    got[0].float().sum()  # (loads its kernels)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    size = got[0].numel() * got[0].element_size()
    address, total = got[0].data_ptr(), got[0].float().sum()
    del got
    with torch.cuda.stream(side):
        again = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() != address
    torch.cuda.synchronize()
    assert not total.isnan()
