"""What the calls refuse of a route of 8-bit weights (no GPU)."""
from __future__ import annotations

import ctypes

import pytest

import moe_expert_lora_amd as ml
from tests.test_fp8_abi import GEMM, LAYER, P, _layer_routes, _refused


@pytest.fixture(scope="module")
def lib():
    return ml.load()


@pytest.mark.parametrize("fast", [-1, 2, 1 << 30])
def test_sums_are_fast_or_not(lib, fast):
    r = ml.Fp8Route(P, P, 4, 300, 100, fast)
    _refused(lib, "mlora_fp8_gemm", {**GEMM, "route": ctypes.byref(r)}, {})
    for name in ("gate", "up", "down"):
        routes = _layer_routes()
        routes[name].contents.fast_sums = fast
        _refused(lib, "mlora_moe_layer", {**LAYER, **routes}, {})


def test_a_route_keeps_its_size():
    """The choice of sums takes what was padding."""
    assert ctypes.sizeof(ml.Fp8Route) == 32 and ml.Fp8Route.fast_sums.offset == 28
