"""What the build makes with and without a PyTorch for ROCm (the compilers stood
in for: their commands are recorded)."""
from __future__ import annotations

import os
import sys

import pytest

from moe_expert_lora_amd import build


@pytest.fixture
def made(monkeypatch, tmp_path):
    """Base names of what a build's commands write, in order."""
    outputs = []

    def run(cmd, verbose):
        out = cmd[cmd.index("-o") + 1]
        with open(out, "wb"):
            pass
        if ".so" in os.path.basename(out):
            outputs.append(os.path.basename(out).replace(".tmp", ""))

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    for name in ("LIB", "PROBE_LIB", "BINDING"):
        path = os.path.join(str(tmp_path), os.path.basename(getattr(build, name)))
        monkeypatch.setattr(build, name, path)
    return outputs


def test_build_without_torch(made, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB
    assert made == ["libmlora.so", "libmlora_probe.so"]
    assert "_native" in capsys.readouterr().err


def test_build_with_a_torch_for_the_cpu(made, monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.version, "hip", None)
    build.build()
    assert made == ["libmlora.so", "libmlora_probe.so"]


def test_build_with_torch(made, monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.version, "hip", "7.0")
    build.build()
    assert made == ["libmlora.so", "libmlora_probe.so", os.path.basename(build.BINDING)]
