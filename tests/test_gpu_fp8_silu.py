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


@pytest.mark.parametrize("top", [448.0, 1.0, 1.5, 3.0, 7.0, 5.0, 0.328125, 1.9921875, 1.1, 1.7])
def test_codes_of_large_gates_are_the_nearest(ml, top):
    """From 20 on 1 + e^-x is 1 in fp32 and silu(x) is x, so silu(x) up is one rounding
    and the codes are known: also half way between two of them, one and two units beside
    that, and where a quotient rounded to fp32 before would fall on it."""
    table = fp8.e4m3_values()
    mid = (table[1:] + table[:-1]) / 2
    top = np.float32(top * 2.0 ** 20)
    near = (mid * np.float64(top) / 448).astype(np.float32)
    near = near[near >= 20]
    rows = [near]
    for _ in range(2):
        rows = [np.nextafter(rows[0], np.float32(0)), *rows, np.nextafter(rows[-1], np.float32(1e9))]
    gate = np.full((3 * len(rows), 128), 20, dtype=np.float32)
    up = np.ones_like(gate)
    for i, r in enumerate(rows):
        gate[3 * i:3 * i + 3, :r.size] = r
    gate[:, 127] = top
    # the same products of a gate and an up, and of both signs
    up[1::3] = -1
    gate[2::3] *= np.float32(1.25)
    up[2::3] = np.float32(0.8)
    x, u = torch.from_numpy(gate).to(DEV), torch.from_numpy(up).to(DEV)
    q = torch.empty((gate.shape[0], 128), dtype=torch.uint8, device=DEV)
    s = torch.empty((1, gate.shape[0]), device=DEV)
    ml.mlora_fp8_quant(x, q, s, up=u)
    codes, _ = fp8.quantise((gate * up).astype(np.float64), 128)
    assert np.array_equal(q.cpu().numpy(), codes)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_codes_of_any_gate(ml, dtype):
    """Those of the fp32 value, which is within 8 roundings (the exponential's two among
    them) of the exact one: the nearest code of it or, across one border, of that much
    less or more."""
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device=DEV).manual_seed(5)
    gate, up = (torch.randn((700, 640), generator=g, device=DEV).mul(2).to(t) for _ in range(2))
    q = torch.empty((700, 640), dtype=torch.uint8, device=DEV)
    s = torch.empty((5, 700), device=DEV)
    ml.mlora_fp8_quant(gate, q, s, up=up)
    v = (fp8.silu(to64(gate)) * to64(up)).reshape(700, 5, 128)
    m = np.abs(v).max(2, keepdims=True)
    got = fp8.e4m3_decode(q.cpu().numpy()).reshape(700, 5, 128)
    slack = 18 * F32  # the value's 8, the largest one's 8, the quotient's own
    ends = [fp8.e4m3_decode(fp8.e4m3_round((v * 448 / m * k).clip(-448, 448)))
            for k in (1 - slack, 1 + slack)]
    assert ((got == ends[0]) | (got == ends[1])).all()
