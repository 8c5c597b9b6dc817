"""Specs and masks as plain values: copied, pickled, compared and hashed by their fields, their C
structs never behind them."""
import copy
import pickle

import pytest

from block_sparse_spatio_attn_b200 import svga

ROTARY = [svga.RotarySpec(4, 2, 5, [10, 11, 11]), svga.RotarySpec(4, 2, 5, (1, 0, 3), False, [0, 2, 1])]
MASKS = [svga.WindowMask(), svga.WindowMask(False, 3, 5, 7)]
PROBLEM = svga.ProblemSpec(2, 3, 4, 5, 64, [0, 1], [1, 2], [0, 1], 1, 64, 64)
WAYS = [copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x)), lambda x: copy.deepcopy([x])[0]]


def c_of(x):
    c = x.c
    if isinstance(x, svga.WindowMask):
        return c.causal, c.window, c.sinks, c.block
    if isinstance(x, svga.RotarySpec):
        order = [c.order[h] for h in range(len(x.order))] if x.order is not None else bool(c.order)
        return c.num_frames, c.grid_h, c.grid_w, tuple(c.pairs), c.interleaved, order, x.rows, x.ordered_heads
    return (c.heads, c.num_frames, c.grid_h, c.grid_w, c.head_dim, [c.head_type[h] for h in range(c.heads)],
            [c.band[h] for h in range(c.heads)], [c.order[h] for h in range(c.heads)], c.anchor_frame0, c.tile_q,
            c.tile_k, c.frame_pad)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("spec", ROTARY + MASKS + [PROBLEM], ids=repr)
def test_copies_and_pickles(spec, way):
    other = way(spec)
    assert other == spec and type(other) is type(spec) and c_of(other) == c_of(spec)
    if spec is not PROBLEM:
        assert hash(other) == hash(spec)


def test_lists_are_taken_as_they_are_then():
    pairs, order = [10, 11, 11], [0, 1]
    spec = svga.RotarySpec(4, 2, 5, pairs, True, order)
    pairs[0], order[1] = 3, 2
    assert spec == svga.RotarySpec(4, 2, 5, (10, 11, 11), True, (0, 1)) and spec.rows == 40 + 22 + 55
    assert c_of(spec)[3] == (10, 11, 11) and c_of(spec)[5] == [0, 1]
    assert len({spec, svga.RotarySpec(4, 2, 5, (10, 11, 11), True, (0, 1))}) == 1


def test_a_module_that_holds_a_spec_is_copied():
    import torch

    class Layer(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.spec, self.mask = ROTARY[1], MASKS[1]

    layer = copy.deepcopy(Layer())
    assert layer.spec == ROTARY[1] and c_of(layer.spec) == c_of(ROTARY[1]) and layer.mask == MASKS[1]
