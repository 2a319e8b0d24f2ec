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


# a route of another class, its address alone, nothing
NOT_W4 = [ml.Fp8Route(P, P, 4, 256, 100), ml.ExpertRoute(), ml.MultiRoute(), P, None]
NOT_FP8 = [ml.W4Route(P, P, None, 4, 256, 100, 64, ml.MLORA_BF16), ml.ExpertRoute(), P, None]


@pytest.mark.parametrize("route", NOT_W4, ids=lambda r: type(r).__name__)
def test_4_bit_products_take_4_bit_routes(route):
    with pytest.raises(TypeError, match="route must be a W4Route"):
        ml.mlora_w4_gather_gemv(route, None, None)


@pytest.mark.parametrize("route", NOT_FP8, ids=lambda r: type(r).__name__)
def test_8_bit_calls_take_8_bit_routes(route):
    with pytest.raises(TypeError, match="route must be a Fp8Route"):
        ml.mlora_fp8_gemm(route, None, None, None)
    right = ml.Fp8Route(P, P, 4, 256, 100)
    for i, name in enumerate(("gate", "up", "down")):
        routes = [right] * 3
        routes[i] = route
        with pytest.raises(TypeError, match=name + " must be a Fp8Route"):
            ml.mlora_moe_layer(*routes, None, None, None, 2, None)


def test_weights_too_large(lib):
    """2^30 blocks and more: refused by the size query as by the call."""
    wide = 1 << 20
    assert ml.mlora_fp8_packed_bytes(16, wide, wide) == 0
    assert ml.mlora_fp8_packed_bytes(15, wide, wide) > 0
    for n in (16, 1024):
        r = ml.Fp8Route()
        assert lib.mlora_fp8_pack(P, P, n, wide, wide, 0, P, (1 << 64) - 1, ctypes.byref(r),
                                  None) == ml.MLORA_ERR_INVALID
        _refused(lib, "mlora_fp8_gemm", {**GEMM, "route": ctypes.byref(ml.Fp8Route(P, P, n, wide, wide))},
                 dict(q_rows=4, q_ld=wide + 128, out_ld=wide))


def test_weights_of_another_device(monkeypatch):
    """The tensors are on the current device already; the routes have to be as well."""
    monkeypatch.setattr(ml, "_device", lambda: 0)
    far4 = ml.W4Route(P, P, None, 4, 256, 100, 64, ml.MLORA_BF16)
    near, far = ml.Fp8Route(P, P, 4, 256, 100), ml.Fp8Route(P, P, 4, 256, 100)
    far4.device = far.device = 1
    near.device = 0
    with pytest.raises(ValueError, match="route must be on the current device"):
        ml.mlora_w4_gather_gemv(far4, None, None)
    with pytest.raises(ValueError, match="route must be on the current device"):
        ml.mlora_fp8_gemm(far, None, None, None)
    for i, name in enumerate(("gate", "up", "down")):
        routes = [near] * 3
        routes[i] = far
        with pytest.raises(ValueError, match=name + " must be on the current device"):
            ml.mlora_moe_layer(*routes, None, None, None, 2, None)
