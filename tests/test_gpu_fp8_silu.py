"""GPU tests of silu in the 8-bit rows' quantiser at both ends of its exponential."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8  # noqa: E402
from tests.fp8_cases import F32, close, to64  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def ml():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_lora_amd
    return moe_expert_lora_amd


@pytest.mark.parametrize("lo,hi", [(-90.0, -88.8), (-88.7, -87.4), (-87.3, -86.0), (-40.0, -10.0),
                                   (-1.0, 1.0), (80.0, 90.0), (120.0, 300.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_of_one_range(ml, lo, hi, dtype):
    """Every gate of a row's groups lies in one range (bf16: to half a step of 0.5), so that a lost exponential is a
    lost group; up lifts the products to about 1. Down to -90 the exponential keeps 19
    bits and more (2^-149 against e^-90 = 2^-129.8), a unit of which is 2^-19 of the
    value; with 10 roundings of fp32 that is the error before the code's rounding."""
    rng = np.random.default_rng(int(hi) + 500)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    gate = torch.from_numpy(rng.uniform(lo, hi, (5, 300))).to(DEV).to(t)
    lift = np.exp(min(-lo, 86.0)) if lo < 0 else 1 / hi
    up = torch.from_numpy(rng.uniform(0.5, 2, (5, 300)) * lift).to(DEV).to(t)
    q = torch.empty((5, ml.mlora_fp8_row_width(300)), dtype=torch.uint8, device=DEV)
    s = torch.empty((3, 5), device=DEV)
    ml.mlora_fp8_quant(gate, q, s, up=up)
    want = fp8.silu(to64(gate)) * to64(up)
    got = fp8.rows_of(q.cpu().numpy(), s.cpu().numpy(), 300)
    scale = to64(s).T[:, np.arange(300) // 128]
    before = np.abs(want) * (2.0 ** -19 + 10 * F32)
    close(got, want, np.maximum((np.abs(want) + before) * 2.0 ** -4, scale * 2.0 ** -10) + before)
    top = np.abs(np.pad(want, ((0, 0), (0, 84)))).reshape(5, -1, 128).max(2)
    close(to64(s).T, top / 448, top / 448 * (2.0 ** -19 + 12 * F32))
