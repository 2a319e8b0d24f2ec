"""GPU test of the norm gradients in one workspace, sized for the largest batch."""
from __future__ import annotations

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


@pytest.mark.parametrize("dim,most", [(300, 2100), (2048, 1100), (4096, 600)])
def test_one_workspace_for_every_batch(ml, dim, most):
    """The sums over the tokens have the bits that a workspace of the batch's own size
    gives, and nothing behind that size is written."""
    g = torch.Generator(device=DEV).manual_seed(dim)
    rows = [torch.randn((most, dim), generator=g, device=DEV).to(torch.bfloat16) for _ in range(3)]
    w = 1 + 0.1 * torch.randn(dim, generator=g, device=DEV)
    whole = torch.empty(ml.mlora_block_norm_backward_workspace_bytes(most, dim), dtype=torch.uint8,
                        device=DEV)
    for t in (most, most - 1, most // 2 + 1, most // 2, 513, 512, 257, 256, 65, 5, 1):
        if t > most:
            continue
        need = ml.mlora_block_norm_backward_workspace_bytes(t, dim)
        got = []
        for ws in (whole, torch.empty(need, dtype=torch.uint8, device=DEV)):
            ws.fill_(0xff)
            d_w = torch.full((dim,), 7.0, device=DEV)
            ml.mlora_block_norm_backward(rows[0][:t], d_r=rows[1][:t], d_x=rows[2][:t],
                                         d_x_weight=d_w, x_weight=w, workspace=ws)
            got.append(d_w)
        assert (whole[need:] == 0xff).all(), t
        assert torch.equal(*got) and got[0].isfinite().all(), t
