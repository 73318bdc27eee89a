"""Caps that are refused (no GPU): the tanh's error is a part of the cap, which bounds it."""

import pytest

from test_span_abi_cpu import BAD, ODD, P, lib, paged, span  # noqa: F401

LARGEST = 16384.0


@pytest.mark.parametrize("cap", [1e-3, 30.0, 1e4, LARGEST])
def test_caps_that_are_taken(lib, cap):  # noqa: F811
    for entry in ("fa_span_fwd", "fa_span_bwd"):
        assert span(lib, entry, cap=cap, q=P + 4) == ODD
    assert paged(lib, cap=cap, q=P + 4) == ODD


@pytest.mark.parametrize("cap", [LARGEST + 1, 1e5, 1e30, 3e38])
def test_caps_beyond_what_the_tanh_holds(lib, cap):  # noqa: F811
    for entry in ("fa_span_fwd", "fa_span_bwd"):
        assert span(lib, entry, cap=cap, q=P + 4) == BAD
    assert paged(lib, cap=cap, q=P + 4) == BAD
