"""The native binding belongs to one Python and one PyTorch: no GPU needed."""
import os
import sysconfig
from types import SimpleNamespace

import pytest
import torch

from io_aware_exact_35_b200 import build, fa


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """The outputs of the compiler calls, which write empty files into a folder."""
    made = []

    def run(cmd, **kw):
        made.append(cmd[cmd.index("-o") + 1])
        open(made[-1], "w").close()
        return SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "LIBDIR", str(tmp_path))
    return made


@pytest.mark.parametrize("what", ["torch", "python"])
def test_another_version_has_a_binding_of_its_own(compiled, monkeypatch, what):
    first = build.build_binding()
    assert os.path.exists(first) and len(compiled) == 1
    assert build.build_binding() == first and len(compiled) == 1
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "99.1.0")
    else:
        monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-x86_64-linux-gnu")
    second = build.build_binding()
    assert len(compiled) == 2 and second != first and os.path.exists(second)


def test_a_binding_for_another_version_is_not_loaded(compiled, monkeypatch):
    build.build_binding()
    monkeypatch.setattr(torch, "__version__", "99.1.0")
    monkeypatch.setattr(fa, "_native_module", None)
    with pytest.raises(RuntimeError, match="is missing: build it"):
        fa.native()
