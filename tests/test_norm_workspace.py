"""Workspace of the norm gradients (no GPU): one of a batch's size does for every
smaller batch, as a program that keeps one buffer needs it."""
from __future__ import annotations

import ctypes

import pytest

import moe_expert_lora_amd as ml
from tests.test_fp8_abi import CAPACITY, P

# widths at both ends of each number of threads a row
DIMS = [1, 300, 512, 513, 1024, 1025, 2048, 2049, 4096, 4097, 8192, 8193, 16384]
TOKENS = list(range(1, 4200)) + [2 ** i + d for i in range(13, 30) for d in (-1, 0, 1)]


@pytest.mark.parametrize("dim", DIMS)
def test_grows_with_the_tokens(dim):
    need = ml.load().mlora_block_norm_backward_workspace_bytes
    sizes = [need(t, dim) for t in TOKENS]
    assert sizes[0] > 0 and sizes == sorted(sizes)


@pytest.mark.parametrize("tokens,dim", [(512, 2048), (600, 2048), (1025, 4096)])
def test_a_smaller_workspace_is_refused(tokens, dim):
    lib = ml.load()
    b = ml.NormBlock(residual=P, residual_ld=dim, x_weight=P, dtype=ml.MLORA_BF16,
                     w_dtype=ml.MLORA_F32, dim=dim, n_tokens=tokens, residual_scale=1.0,
                     y_scale=1.0, eps=1e-6)
    need = ml.mlora_block_norm_backward_workspace_bytes(tokens, dim)
    assert lib.mlora_block_norm_backward(
        ctypes.byref(b), P, dim, P, dim, P, dim, None, 0, P, None, None, 0, P, need - 1,
        None) == CAPACITY
