"""make_w4_route without a GPU: where the packed memory comes from and which
tensors it takes, with the library's call and the tensors stood in for."""
from __future__ import annotations

import contextlib
import types

import pytest

import moe_expert_lora_amd as ml

torch = pytest.importorskip("torch")


class Tensor:
    """What make_w4_route asks of a device tensor."""

    is_cuda = True

    def __init__(self, shape, dtype, index=0):
        self.shape, self.dtype = shape, dtype
        self.device = torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def calls(monkeypatch):
    """The pack calls and allocations made, and the stream current at each allocation."""
    seen = types.SimpleNamespace(packs=[], allocations=[], current="current")
    real = ml.load()

    def pack(*args):
        seen.packs.append(args[-1])
        return ml.MLORA_OK

    @contextlib.contextmanager
    def on_stream(stream):
        old, seen.current = seen.current, stream
        yield
        seen.current = old

    def empty(n, dtype, device):
        seen.allocations.append((n, device, seen.current))
        return Tensor((n,), dtype, device.index)

    lib = types.SimpleNamespace(mlora_w4_pack=pack,
                                mlora_w4_packed_bytes=real.mlora_w4_packed_bytes)
    monkeypatch.setattr(ml, "load", lambda: lib)
    monkeypatch.setattr(ml, "_stream_handle", lambda s: "handle of current" if s is None else s)
    monkeypatch.setattr(ml, "_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", on_stream)
    monkeypatch.setattr(torch, "empty", empty)
    return seen


def _args(q=0, scales=0, zeros=0):
    """Tensors of 2 x 48 x 64 in groups of 32, each on the device of that index."""
    return (Tensor((2, 48, 32), torch.uint8, q), Tensor((2, 48, 2), torch.bfloat16, scales),
            None if zeros is None else Tensor((2, 48, 2), torch.uint8, zeros), 64, 32)


def test_packed_memory_is_of_the_stream_that_writes_it(calls):
    """A block of the current stream's could still be in use there while `side`
    writes it, and would go back there while `side` still reads it."""
    route = ml.make_w4_route(*_args(), stream="side")
    nbytes = ml.mlora_w4_packed_bytes(2, 64, 48, 32, ml.MLORA_BF16, True)
    assert calls.allocations == [(nbytes, torch.device("cuda", 0), "side")]
    assert calls.packs == ["side"] and calls.current == "current"
    assert route._keep.shape == (nbytes,)


def test_packed_memory_of_the_current_stream(calls):
    ml.make_w4_route(*_args(zeros=None))
    assert [a[2] for a in calls.allocations] == ["current"]
    assert calls.packs == ["handle of current"]


@pytest.mark.parametrize("where,name", [((1, 1, 1), "q"), ((1, 0, 0), "q"), ((0, 1, 0), "scales"),
                                        ((0, 0, 1), "zeros"), ((0, 1, None), "scales")])
def test_tensors_of_another_device_are_refused(calls, where, name):
    """The pack runs on the current device (0 here)."""
    with pytest.raises(ValueError, match=f"{name} must be on the current device"):
        ml.make_w4_route(*_args(*where))
    assert not calls.packs and not calls.allocations


@pytest.mark.parametrize("k_in,group,q,scales", [
    (264, (1 << 32) + 64, (1, 48, 132), (1, 48, 1)),    # as 64: five scales a row, one is there
    ((1 << 32) + 64, 1 << 20, (1, 1, (1 << 31) + 32), (1, 1, (1 << 12) + 1)),
    (64, 64, (1, (1 << 32) + 8, 32), (1, (1 << 32) + 8, 1)),
    (64, 64, ((1 << 32) + 1, 8, 32), ((1 << 32) + 1, 8, 1))])
def test_sizes_past_32_bits_are_refused(calls, k_in, group, q, scales):
    """Not taken by their low halves."""
    with pytest.raises(ValueError, match="out of range"):
        ml.make_w4_route(Tensor(q, torch.uint8), Tensor(scales, torch.bfloat16), None, k_in, group)
    assert not calls.packs and not calls.allocations


def test_size_queries_past_32_bits():
    for args in ((1, 64, 64, (1 << 32) + 64), (1, (1 << 32) + 64, 64, 64),
                 (1, 64, (1 << 32) + 64, 64), ((1 << 32) + 1, 64, 64, 64)):
        with pytest.raises(ValueError, match="out of range"):
            ml.mlora_w4_packed_bytes(*args, ml.MLORA_BF16, False)
    with pytest.raises(ValueError, match="out of range"):
        ml.mlora_moe_sort_workspace_bytes(100000, (1 << 32) + 4)
