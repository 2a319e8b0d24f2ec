"""GPU tests of the 4-bit products at the ends of their ranges of sizes."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def ml():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_lora_amd
    return moe_expert_lora_amd


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [512, (1 << 20) + 128, 2 ** 31 - 128])
def test_one_group_longer_than_a_row(ml, dtype, group):
    """A group of any length above k_in is one group: the same bits as 384."""
    k, n, rows = 264, 50, 7
    rng = np.random.default_rng(1)
    q = torch.from_numpy(rng.integers(0, 256, size=(2, n, k // 2), dtype=np.uint8)).to(DEV)
    s = torch.from_numpy(rng.random((2, n, 1)) + 0.5).to(DEV).to(dtype)
    z = torch.from_numpy(rng.integers(0, 16, size=(2, n, 1), dtype=np.uint8)).to(DEV)
    x = torch.from_numpy(rng.normal(size=(rows, k))).to(DEV).to(dtype)
    ids = torch.from_numpy(rng.integers(0, 2, size=rows).astype(np.int32)).to(DEV)
    outs = []
    for g in (384, group):
        route = ml.make_w4_route(q, s, z, k, g)
        outs.append(torch.empty((rows, n), dtype=dtype, device=DEV))
        ml.mlora_w4_gather_gemv(route, x, outs[-1], ids)
    assert bool((outs[0] != 0).any())
    assert torch.equal(outs[0], outs[1])
