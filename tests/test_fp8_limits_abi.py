"""Refusals of sizes and of memory that two outputs share (no GPU): 8-bit products,
the layer of a few tokens, the norms around a block."""
from __future__ import annotations

import ctypes

import pytest

import moe_expert_lora_amd as ml
from tests.test_fp8_abi import GEMM, LAYER, P, QUANT, _layer_routes, _refused

WIDE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return ml.load()


def test_products_of_more_than_32_bit_offsets(lib):
    r = ml.Fp8Route(P, P, 4, 300, 100)
    base = {**GEMM, "route": ctypes.byref(r)}
    # the last row's end, one byte past what 32 bits count, and a stride alone
    _refused(lib, "mlora_fp8_gemm", base, dict(q_rows=(1 << 32) // 384 + 1))
    _refused(lib, "mlora_fp8_gemm", base, dict(q_rows=2, q_ld=(1 << 32) - 256))
    _refused(lib, "mlora_fp8_gemm", base, dict(q_rows=1, q_ld=1 << 32))
    one = ml.Fp8Route(P, P, 1, 128, WIDE)
    n = (1 << 30) - 1
    _refused(lib, "mlora_fp8_gemm", base,
             dict(route=ctypes.byref(one), q_rows=100, q_ld=128, n=n, out_ld=WIDE, offsets=P))


def test_quantising_more_than_32_bits_of_groups(lib):
    _refused(lib, "mlora_fp8_quant", QUANT,
             dict(n=(1 << 30) - 1, k=WIDE, x_ld=WIDE, q_ld=WIDE + 128))


def test_layers_too_wide_for_their_rows(lib):
    # 16 tokens of 64 experts: 1024 rows of 6 bytes a column
    routes = _layer_routes((64, 256, WIDE), (64, 256, WIDE), (64, WIDE, 256))
    _refused(lib, "mlora_moe_layer", {**LAYER, **routes},
             dict(n=16, k=64, logits_ld=64))
    assert ml.mlora_moe_layer_workspace_bytes(16, 64, 64, 256, WIDE) == 0
    assert ml.mlora_moe_layer_workspace_bytes(16, 64, 4, 256, WIDE) > 0


NORM = ml.NormBlock(residual=P, residual_ld=64, y=P, y_ld=64, x_weight=P, y_weight=P, gate=P,
                    gate_ld=64, gate_form=3, dtype=ml.MLORA_F32, w_dtype=ml.MLORA_F32, dim=64,
                    n_tokens=5, residual_scale=1.0, y_scale=1.0, weight_offset=0.0, eps=1e-6)
OUT = dict(d_residual=1, d_y=2, d_x_weight=3, d_y_weight=4, d_gate=5)


@pytest.mark.parametrize("a", OUT)
@pytest.mark.parametrize("b", OUT)
def test_norm_outputs_are_apart(lib, a, b):
    if a >= b:
        return
    at = {n: P * i for n, i in OUT.items()}
    at[a] = at[b]
    args = [ctypes.byref(NORM), P * 8, 64, P * 9, 64, at["d_residual"], 64, at["d_y"], 64,
            at["d_x_weight"], at["d_y_weight"], at["d_gate"], 64, P * 10, 1 << 40, None]
    assert lib.mlora_block_norm_backward(*args) == ml.MLORA_ERR_INVALID
    assert "same memory" in lib.mlora_last_error().decode()


def test_layer_workspace_grows_with_the_tokens():
    """One of 16 tokens' size does for fewer (the example's decode relies on it)."""
    for E, k, dim, hidden in [(128, 8, 2048, 768), (12, 3, 1000, 365), (68, 6, 154, 1153),
                              (1024, 64, 40, 24), (1, 1, 1, 1), (21, 4, 129, 1873)]:
        sizes = [ml.mlora_moe_layer_workspace_bytes(t, E, k, dim, hidden) for t in range(1, 17)]
        assert sizes == sorted(sizes)
