"""Refusals at the far end of the arguments' ranges, on the host."""
import ctypes

import pytest

from block_sparse_spatio_attn_b200 import svga

SHAPE = 2
A, Z = 1 << 20, 1 << 30  # addresses that are never touched


@pytest.fixture(scope="module")
def lib():
    from block_sparse_spatio_attn_b200 import build
    build.build()
    return svga.load()


def view(data=A, sb=6400, sh=640, st=64):
    return svga.View(data, sb, sh, st)


@pytest.mark.parametrize("first", [2**63 - 1, 2**63 - 10, 2**62, 2**32, 2**31, 91])
def test_a_first_token_whose_sum_with_the_tokens_wraps_is_refused(lib, first):
    """10 tokens from there on pass the 100 of the grid, also where first + 10 wraps to below 0."""
    spec = svga.RotarySpec(10, 2, 5, (10, 11, 11))
    rc = lib.svga_rotary(ctypes.byref(view()), ctypes.byref(view(Z)), 2, 10, 10, 64, 0, ctypes.byref(spec.c), A, None,
                         first, 0, None, None)
    assert rc == SHAPE and "pass the grid" in lib.svga_last_error().decode(), (rc, lib.svga_last_error())
