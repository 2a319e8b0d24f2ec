"""GPU tests of the 8-bit products in every form of the launch plan, against fp64: bf16
and float32 results, fp32 sums and fast ones, one weight and spans of many (skewed, rows
through sorted ids, rows in no span)."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8  # noqa: E402
from tests.fp8_cases import F32, U, close, product_error, to64, weights  # noqa: E402
from tests.fp8_forms import FORMS  # noqa: E402
from tests.test_gpu_fp8 import dev, rows_in, spans, whole  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ml():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_lora_amd
    return moe_expert_lora_amd


@pytest.mark.parametrize("skew", [False, True])
@pytest.mark.parametrize("E,N,K,n,full,fast", FORMS)
def test_form(ml, E, N, K, n, full, fast, skew):
    """Tolerance: K products and the blocks' sums in fp32, then one rounding; of fast sums
    what the 8-bit instruction cuts off besides."""
    rng = np.random.default_rng(N + n + skew)
    one = E == 0
    w, ws = weights(rng, max(E, 1), N, K)
    top_k = 2 if skew else 1
    codes, qs = fp8.quantise(rng.normal(0, 1, (n // top_k, K)), whole(K))
    qs = qs.astype(np.float32)
    lead, behind = (3, 5) if skew else (0, 0)
    off = None if one else spans(rng, n, E, lead, behind, skew)
    order = None
    if skew:
        order = rng.permutation(n).astype(np.int32)
        order[::17] = -1
        order[5::29] = n + 3
    base = rng.normal(0, 1, (n, N)).astype(np.float32)
    q, s = rows_in(ml, codes), dev(qs)
    off_d = None if off is None else dev(off)
    ids = None if order is None else dev(order)
    expanded, values = fp8.expand(w, ws), fp8.rows_of(codes, qs, K)
    ref, mag = fp8.products(expanded, values, off, order, top_k, base)
    inner = mag * (K + -(-K // 128) + 4) * F32
    for dtype, short in (("bf16", False), ("f32", False), ("bf16", True)):
        route = ml.make_fp8_route(dev(w).view(torch.float8_e4m3fn), dev(ws), fast_sums=short)
        out = dev(base).to(TORCH[dtype])
        before = to64(out)
        ml.mlora_fp8_gemm(route, q, s, out, off_d, ids, top_k)
        err = product_error(ref, mag, K, "bf16") if short else \
            inner + (np.abs(ref) + inner) * U[dtype]
        close(to64(out), np.where(mag > 0, ref, before), np.where(mag > 0, err, 0.0),
              (dtype, short))
