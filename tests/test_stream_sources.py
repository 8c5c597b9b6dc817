"""Rules of the streaming kernels that no call can show on a healthy GPU, held to their sources."""
import os
import re

import pytest

from block_sparse_spatio_attn_b200 import build

KERNELS = ["rotary.cu", "decode.cu", "window_fwd.cu", "window_bwd.cu"]


def source(name):
    return open(os.path.join(build.CSRC, name)).read()


@pytest.mark.parametrize("name", KERNELS)
def test_a_status_word_keeps_its_first_failure(name):
    """A later failure (a wait that ran out, say) must not replace an earlier one: every report goes
    through the one function, which writes only over 0."""
    text = source(name)
    assert "report(" in text
    assert not re.search(r"atomic(Exch|CAS)|status\s*=\s*\(int32_t\)|\*\s*p\.(s\.)?status", text)
    body = re.search(r"void report\(int32_t \*status, int32_t code\)\s*\{(.*?)\n\}", source("svga_device.cuh"), re.S)
    assert body and "atomicCAS(status, 0, code)" in body.group(1)
