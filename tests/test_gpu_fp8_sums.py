"""GPU tests of how the 8-bit products add: in fp32 whatever the result's type, or,
where a route asks for it, as the 8-bit matrix instruction does.

Inputs. Of eight neighbouring products one is large and cancels exactly against the
next eight's; the other seven, 0.125 to 0.42 times the block's scales, are all the sum
there is. The large one is 448 * 32, between 2^13 and 2^14, so the instruction, which
keeps what is above 2^-13 of its power of two, loses the others.

Tolerance. fp32 sums of K products and their blocks are within (K + blocks + 4) 2^-24 of
the magnitudes' sum, then one rounding. The large products add 2 * 448 * 32 to the
magnitudes for each 16 columns: a bound of 0.45 for them at K = 256, 1.1 at K = 640,
against a sum of 14 * 0.24 = 3.4, so the loss is far outside.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8  # noqa: E402
from tests.fp8_cases import F32, U, close, product_error, to64, weights  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ml():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_lora_amd
    return moe_expert_lora_amd


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def cancelling(rng, E, N, K, n):
    """Codes of weights [E, N, K] and rows [n, K], and their scales."""
    w, q = rng.uniform(0.5, 0.8, (E, N, K)), rng.uniform(0.25, 0.5, (n, K))
    w[..., ::8], q[..., ::8] = 32, 448
    w[..., 8::16] = -32
    sign = rng.choice([-1.0, 1.0], (n, 1))
    blocks = -(-K // 128)
    ws = rng.uniform(0.5, 2, (E, -(-N // 128), blocks)).astype(np.float32)
    return fp8.e4m3_round(w), ws, fp8.e4m3_round(q * sign), \
        rng.uniform(0.5, 2, (blocks, n)).astype(np.float32)


# E, N, K, rows: waves of 16 rows, tiles of 32, 64, 128 and 256 rows
SIZES = [(1, 64, 256, 20), (40, 260, 384, 1300), (64, 900, 640, 2560), (2, 2300, 256, 8300),
         (20, 2500, 640, 5200)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,N,K,n", SIZES)
def test_sums_are_fp32(ml, E, N, K, n, dtype):
    rng = np.random.default_rng(N + n)
    w, ws, q, qs = cancelling(rng, E, N, K, n)
    off = np.linspace(0, n, E + 1).astype(np.int32)
    rows = torch.zeros((n, ml.mlora_fp8_row_width(K)), dtype=torch.uint8, device=DEV)
    rows[:, :K] = dev(q)
    ref, mag = fp8.products(fp8.expand(w, ws), fp8.rows_of(q, qs, K), off, None, 1,
                            np.zeros((n, N)))
    out = {}
    for fast in (False, True):
        route = ml.make_fp8_route(dev(w), dev(ws), fast_sums=fast)
        out[fast] = torch.full((n, N), 7.0, dtype=TORCH[dtype], device=DEV)
        ml.mlora_fp8_gemm(route, rows, dev(qs), out[fast], dev(off))
    err = mag * (K + -(-K // 128) + 4) * F32
    close(to64(out[False]), ref, err + (np.abs(ref) + err) * U[dtype])
    if dtype == "f32":
        assert torch.equal(out[True], out[False])
    else:
        close(to64(out[True]), ref, product_error(ref, mag, K, "bf16"))


@pytest.mark.parametrize("e", [-110, -118, -126])
@pytest.mark.parametrize("E,N,K,n", SIZES[:4])
def test_rows_of_small_values(ml, E, N, K, n, e):
    """Rows of 2^e: their scales times the weights' 2^-12 or so fall below fp32's smallest
    normal value, and enter to half of 2^-149 times the block's products."""
    rng = np.random.default_rng(n)
    w, ws = weights(rng, E, N, K)
    x = torch.from_numpy(rng.normal(0, 1, (n, K)) * 2.0 ** e).to(DEV).float()
    q = torch.zeros((n, ml.mlora_fp8_row_width(K)), dtype=torch.uint8, device=DEV)
    s = torch.empty((-(-K // 128), n), device=DEV)
    ml.mlora_fp8_quant(x, q, s)
    off = np.linspace(0, n, E + 1).astype(np.int32)
    out = torch.empty((n, N), device=DEV)
    ml.mlora_fp8_gemm(ml.make_fp8_route(dev(w), dev(ws)), q, s, out, dev(off))
    codes, qs = q.cpu().numpy(), s.cpu().numpy()
    ref, mag = fp8.products(fp8.expand(w, ws), fp8.rows_of(codes, qs, K), off, None, 1,
                            np.zeros((n, N)))
    # the magnitudes without scales
    _, units = fp8.products(fp8.expand(w, np.ones_like(ws)), fp8.rows_of(codes, np.ones_like(qs), K),
                            off, None, 1, np.zeros((n, N)))
    tiny = 2.0 ** -150
    err = mag * (K + -(-K // 128) + 4) * F32 + units * tiny + (-(-K // 128) + 1) * tiny
    close(to64(out), ref, err + (np.abs(ref) + err) * U["f32"])


def test_packing_asks_for_fp32(ml):
    w, s = torch.zeros((1, 8, 8), dtype=torch.uint8, device=DEV), torch.ones((1, 1, 1), device=DEV)
    assert ml.make_fp8_route(w, s).fast_sums == 0
    assert ml.make_fp8_route(w, s, fast_sums=True).fast_sums == 1


def test_routes_name_their_device(ml):
    w, s = torch.zeros((1, 8, 8), dtype=torch.uint8, device=DEV), torch.ones((1, 1, 1), device=DEV)
    assert ml.make_fp8_route(w, s).device == torch.cuda.current_device()
    route = ml.make_w4_route(w, torch.ones((1, 8, 1), device=DEV), None, 16, 32)
    assert route.device == torch.cuda.current_device()
