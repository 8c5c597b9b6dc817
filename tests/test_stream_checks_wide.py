"""Refusals at the far end of the arguments' ranges, on the host."""
import ctypes

import pytest
import torch

from block_sparse_spatio_attn_b200 import svga

ARG, SHAPE = 1, 2
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


def rejected(fn, status, words):
    with pytest.raises(svga.SvgaError) as e:
        fn()
    assert e.value.status == status and words in str(e.value), str(e.value)


def test_flags_that_32_bits_would_cut_to_0_are_refused():
    rejected(lambda: svga.WindowMask(causal=2**32), 2, "does not fit 32 bits")
    rejected(lambda: svga.RotarySpec(1, 2, 5, (1, 1, 1), interleaved=2**32), 2, "does not fit 32 bits")
    spec = svga.RotarySpec(1, 2, 5, (10, 11, 11))
    x, t = torch.zeros(1, 2, 10, 64, dtype=torch.bfloat16), torch.zeros(spec.table_shape)
    for inverse in (2**32, -2**31 - 1, 2**40 + 1):
        rejected(lambda: svga.svga_rotary(x, x, spec, t, inverse=inverse), 1, "inverse: ")


def test_workspace_size_of_tensors_that_no_call_takes():
    q = torch.zeros(1, 2, 3, 64, dtype=torch.float16)
    size = svga.svga_window_attention_size
    for k in (q[..., :32], q.expand(2, 2, 3, 64), q.bfloat16()):
        rejected(lambda: size(q, k, svga.WindowMask()), 2, "k has shape")
    wide = q.expand(2**32 + 1, 2, 3, 64)  # ctypes would make it a batch of 1
    rejected(lambda: size(wide, wide, svga.WindowMask()), 2, "does not fit 32 bits")
    assert size(q, q[:, :1], svga.WindowMask())["bwd_bytes"] > 0


def test_pages_that_keys_and_values_would_both_be_written_to_are_refused(lib):
    """Decoding from one tensor as K and V is fine; appending writes both."""
    c = svga.PagedCacheC(Z, Z, 4, 2, 16, 64, 0, 2, 2, A, A, None)
    v = ctypes.byref(view())
    rc = lib.svga_cache_append(v, v, 3, None, ctypes.byref(c), None, None, None)
    assert rc == ARG and "start together" in lib.svga_last_error().decode(), (rc, lib.svga_last_error())
    assert lib.svga_cache_append(v, v, 0, None, ctypes.byref(c), None, None, None) == 0
