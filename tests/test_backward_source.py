"""The models of the backward kernel's hand-offs (test_backward_order.py) against its source: the
stages and the arrivals a phase that they assume are the kernel's, and they hold with its numbers of
warps."""
import inspect
import os
import random
import re

import pytest

from block_sparse_spatio_attn_b200 import build
from tests import test_backward_order as models

TEXT = open(os.path.join(build.CSRC, "window_bwd.cu")).read()


def part(begin, end):
    i = TEXT.index(begin)
    return TEXT[i:TEXT.index(end, i)]


DKDV = part("__device__ __forceinline__ void dkdv_cta(", "bwd_join_kernel(")
DQ = part("__device__ __forceinline__ void dq_cta(", "bwd_kernel(")


def constant(name):
    return int(re.search(rf"\b{name} = (\d+)", TEXT).group(1))


def arrivals(text):
    return {name: int(n) for name, n in re.findall(r"mbar_init\(smem_u32\(&bar->(\w+)(?:\[i\])?\), (\d+)\)", text)}


def default(model, name):
    return inspect.signature(model).parameters[name].default


def test_stages_are_the_kernels():
    assert default(models.dkdv_cta, "QS") == constant("kQStages")
    assert default(models.dkdv_cta, "OS") == constant("kOStages")
    assert default(models.dq_cta, "KS") == constant("kKStages")
    assert default(models.dq_cta, "VS") == constant("kVStages")


def test_arrivals_are_the_kernels():
    warps = constant("kThreads") // 32 - 4  # of both softmax groups
    one = dict.fromkeys(["kv_full", "q_full", "q_empty", "o_full", "st_full", "st_empty", "s_full", "dp_full",
                         "zero_req", "zero_done", "drain"], 1)
    # o_empty: dV and dP of a step; acc_done: both issuers; the groups' own barriers: their warps
    assert arrivals(DKDV) == {**one, "o_empty": 2, "acc_done": 2, "p_ready": warps // 2, "ds_ready": warps // 2}
    one = dict.fromkeys(["q_full", "k_full", "k_empty", "v_full", "v_empty", "s_full", "dp_full", "dq_done", "drain",
                         "zero_done"], 1)
    assert arrivals(DQ) == {**one, "a_ready": warps, "s_free": warps, "dp_free": warps, "ds_ready": warps}


def test_who_completes_what():
    """The commits and arrivals behind each product and step, by number."""
    def count(text, what):
        return len(re.findall(what, text))
    for name in ("q_empty", "st_empty", "dp_full"):
        assert count(DKDV, rf"mma_commit\(smem_u32\(&bar->{name}\b") == 1, name
    assert count(DKDV, r"mma_commit\(smem_u32\(&bar->o_empty\b") == 2
    for name in ("p_ready", "ds_ready"):
        assert count(DKDV, rf"if \(lane == 0\) mbar_arrive\(smem_u32\(&bar->{name}\[wg\]\)\)") == 1, name
    for name in ("s_full", "dq_done", "k_empty", "dp_full", "v_empty"):
        assert count(DQ, rf"mma_commit\(smem_u32\(&bar->{name}\b") == 1, name
    for name in ("s_free", "dp_free", "ds_ready"):
        assert count(DQ, rf"if \(lane == 0\) mbar_arrive\(smem_u32\(&bar->{name}\)\)") == 1, name


@pytest.mark.parametrize("seed", range(2))
def test_models_with_the_kernels_numbers(seed):
    rng = random.Random(seed)
    warps = constant("kThreads") // 32 - 4
    for _ in range(150):
        assert models.dq_cta(rng.randint(1, 12), rng.random() < 0.5, rng, warps, constant("kKStages"),
                             constant("kVStages")) == []
        n_blk, group = rng.randint(1, 5), rng.randint(1, 4)
        first = rng.randint(0, n_blk * group - 1)
        steps = rng.randint(1, n_blk * group - first)
        ragged = n_blk - 1 if rng.random() < 0.6 else -1
        assert models.dkdv_cta(n_blk, group, first, steps, ragged, rng, warps // 2, constant("kQStages"),
                               constant("kOStages")) == []
