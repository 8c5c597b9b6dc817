"""The compiled Python binding belongs to one torch and one Python: another makes it stale, and is
refused when it is loaded all the same."""
import os

import pytest

from block_sparse_spatio_attn_b200 import build, svga


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """The build with a recorder in place of the compiler; what it would have compiled."""
    build.build()
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return type("Done", (), {"returncode": 0, "stdout": "", "stderr": ""})()

    binding = tmp_path / "_binding.so"
    binding.write_bytes(b"")
    monkeypatch.setattr(build, "BINDING", str(binding))
    monkeypatch.setattr(build, "BINDING_FOR", str(tmp_path / "binding_for.txt"))
    monkeypatch.setattr(build.subprocess, "run", run)
    return commands


def test_a_binding_for_another_torch_is_built_again(compiled, monkeypatch):
    with open(build.BINDING_FOR, "w") as f:
        f.write(build.binding_for())
    build._build_binding(False, False)
    assert compiled == []
    import torch
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    build._build_binding(False, False)
    assert len(compiled) == 1 and any(".other" in x for x in compiled[0])
    build._build_binding(False, False)
    assert len(compiled) == 1
    os.remove(build.BINDING_FOR)  # not known what it was built for
    build._build_binding(False, False)
    assert len(compiled) == 2


def test_a_binding_for_another_torch_is_refused(monkeypatch):
    build.build()
    svga._binding()
    import torch
    monkeypatch.setattr(svga, "_native", None)
    monkeypatch.setattr(torch, "__version__", "0.0")
    with pytest.raises(svga.SvgaError) as e:
        svga._binding()
    assert e.value.status == 6 and "torch 0.0" in str(e.value)
