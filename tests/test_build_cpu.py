"""What the build makes, and when it makes it again, without running a compiler."""
import os

import pytest

from linear_attention_08_b200 import build as kbuild
from linear_attention_08_b200 import kda


@pytest.fixture
def made(tmp_path, monkeypatch):
    """A build in an empty folder whose compilers only leave files; the names made, in order."""
    made = []

    def compiled(src, verbose):
        made.append(os.path.basename(src))
        return src

    def linked(cmd):
        made.append("libkda.so")
        open(cmd[cmd.index("-o") + 1], "w").close()

    def bound():
        made.append("_binding.so")
        for p in (kbuild.BINDING, kbuild.BINDING_TORCH):
            with open(p, "w") as f:
                f.write(kbuild._torch_version())

    monkeypatch.setattr(kbuild, "BUILD", str(tmp_path))
    for name in ("LIB", "BINDING", "BINDING_TORCH"):
        monkeypatch.setattr(kbuild, name, str(tmp_path / os.path.basename(getattr(kbuild, name))))
    monkeypatch.setattr(kbuild, "_compile", compiled)
    monkeypatch.setattr(kbuild.subprocess, "check_call", linked)
    monkeypatch.setattr(kbuild, "_build_binding", bound)
    return made


def test_the_library_needs_no_pytorch(made, monkeypatch):
    monkeypatch.setattr(kbuild, "_torch_version", lambda: None)
    assert kbuild.build() == kbuild.LIB
    assert made[-1] == "libkda.so" and "_binding.so" not in made
    assert kbuild.up_to_date()


def test_the_binding_can_be_left_out(made):
    kbuild.build(binding=False)
    assert "_binding.so" not in made
    assert kbuild.up_to_date(binding=False) and not kbuild.up_to_date()
    n = len(made)
    kbuild.build()                                   # the library is there already
    assert made[n:] == ["_binding.so"] and kbuild.up_to_date()


def test_another_pytorch_makes_the_binding_again(made, monkeypatch):
    kbuild.build()
    assert kbuild.up_to_date()
    monkeypatch.setattr(kbuild, "_torch_version", lambda: "0.0.1")
    n = len(made)
    assert not kbuild.up_to_date()
    kbuild.build()
    assert made[n:] == ["_binding.so"]


def test_a_binding_for_another_pytorch_is_not_used(monkeypatch):
    monkeypatch.setattr(kda, "_native_module", None)
    monkeypatch.setattr(kda.torch, "__version__", "0.0.1")
    with pytest.raises(ImportError, match="built for PyTorch"):
        kda._native()


def test_the_version_is_found_without_importing_pytorch():
    import torch
    assert kbuild._torch_version() == str(torch.__version__)
