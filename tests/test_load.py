"""Loading the library where torch, or parts of it, are not there."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest

import moe_expert_lora_amd as ml

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def unloaded(monkeypatch):
    for name, value in (("_lib", None), ("_raw_stream", None), ("_device", None)):
        monkeypatch.setattr(ml, name, value)
    return monkeypatch


def _host_functions():
    tables = ml.mlora_pack_expert_tables([0, 2], [16, 32], [48, 64], np.ones(2, np.float32))
    assert tables[3] == 3 and tables[0].tolist() == [16, 0, 32]
    assert ml.mlora_moe_sort_workspace_bytes(100000, 128) > 0


def test_host_functions_with_a_torch_for_the_cpu(unloaded):
    """A torch built without device support has no such names in torch._C."""
    torch = pytest.importorskip("torch")
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        unloaded.delattr(torch._C, name, raising=False)
    _host_functions()


def test_current_stream_without_the_short_forms(unloaded):
    """Device calls then take the stream by torch's public calls."""
    torch = pytest.importorskip("torch")
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        unloaded.delattr(torch._C, name, raising=False)
    stream = type("Stream", (), {"cuda_stream": 77})
    unloaded.setattr(torch.cuda, "current_device", lambda: 3)
    unloaded.setattr(torch.cuda, "current_stream", lambda d: stream if d == 3 else None)
    assert ml._stream_handle(None) == 77


def test_host_functions_without_torch():
    code = ("import sys; sys.modules['torch'] = None\n"
            "import moe_expert_lora_amd as ml\n"
            "print(ml.mlora_m_tile(), ml.mlora_moe_sort_workspace_bytes(100000, 128))")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                         timeout=120)
    assert out.returncode == 0, out.stderr
    assert out.stdout.split()[0] == str(ml.mlora_m_tile())
