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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,experts,k,n,group,zeros", [
    (1, 1, 64, 40, 64, True), (70, 1, 520, 100, 128, False), (2500, 1, 72, 35, 32, True),
    (90, 1, 264, 17001, 64, False),                       # one expert, and ids all the same
    (1, 1024, 264, 40, 64, True), (1023, 1024, 72, 65, 32, False),
    (1024, 1024, 136, 33, 128, True), (5000, 1024, 40, 50, 32, False),   # the most experts
    (3, 1, 1 << 20, 33, 128, True), (2, 2, 1 << 20, 70, 1 << 20, False),  # the longest rows
    (2, 2, 8, 1 << 20, 32, True)])                        # the most columns
def test_ends_of_the_ranges(ml, dtype, rows, experts, k, n, group, zeros):
    """The tolerance per element is the probabilistic bound of 4 K roundings on
    partial sums of at most 15 sum |x| |s|, and half a bf16 step."""
    g = torch.Generator(device=DEV).manual_seed(rows + experts)
    groups = -(-k // group)
    q = torch.randint(0, 256, (experts, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = ((torch.rand((experts, n, groups), generator=g, device=DEV) + 0.5) * k ** -0.5).to(dtype)
    z = torch.randint(0, 16, (experts, n, groups), generator=g, device=DEV,
                      dtype=torch.uint8) if zeros else None
    route = ml.make_w4_route(q, s, z, k, group)
    x = torch.randn((rows, k), generator=g, device=DEV).to(dtype)
    ids = torch.randint(0, experts, (rows,), generator=g, device=DEV, dtype=torch.int32)
    ids[torch.rand(rows, generator=g, device=DEV) < 0.1] = -1
    ids[-1] = experts - 1
    out = torch.full((rows, n), 9.0, dtype=dtype, device=DEV)
    ml.mlora_w4_gather_gemv(route, x, out, ids)
    assert not bool(out[ids < 0].any())
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    for e in torch.unique(ids[ids >= 0]).tolist():
        r = torch.nonzero(ids == e).flatten()
        sc = s[e].double().repeat_interleave(group, 1)[:, :k]
        zero = 8.0 if z is None else z[e].double().repeat_interleave(group, 1)[:, :k]
        w = (torch.stack((q[e] & 15, q[e] >> 4), 2).flatten(1).double() - zero) * sc
        xs = x[r].double()
        ref, mag = xs @ w.t(), xs.abs() @ sc.t()
        tol = 10 * (4 * k) ** 0.5 * 2.0 ** -24 * 15 * mag
        assert bool(((out[r].double() - ref).abs() <= tol + half * (ref.abs() + tol)).all()), e


def test_longest_row_past_its_range_is_refused(ml):
    q = torch.zeros((1, 8, (1 << 19) + 4), dtype=torch.uint8, device=DEV)
    with pytest.raises(ml.MloraError):
        ml.make_w4_route(q, torch.ones((1, 8, 1), device=DEV), None, (1 << 20) + 8, 1 << 21)


@pytest.mark.parametrize("dtype,ld", [(torch.bfloat16, 1_073_741_700 // 8 * 8),
                                      (torch.float32, 536_870_700 // 8 * 8)])
@pytest.mark.parametrize("n", [50, 16420])
def test_x_rows_that_span_almost_4_gib(ml, dtype, ld, n):
    """The last row lies just before the 4 GiB that x may span. Both forms (few
    columns, many) give the bits of packed rows."""
    k, rows = 64, 3
    g = torch.Generator(device=DEV).manual_seed(4)
    q = torch.randint(0, 256, (1, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = (torch.rand((1, n, 1), generator=g, device=DEV) + 0.5).to(dtype)
    route = ml.make_w4_route(q, s, None, k, k)
    x = torch.randn((rows, k), generator=g, device=DEV).to(dtype)
    want, got = (torch.empty((rows, n), dtype=dtype, device=DEV) for _ in range(2))
    ml.mlora_w4_gather_gemv(route, x, want)
    flat = torch.empty(2 * ld + 2 * k, dtype=dtype, device=DEV)
    far = flat.as_strided((rows, k), (ld, 1))
    far.copy_(x)
    ml.mlora_w4_gather_gemv(route, far, got)
    assert torch.equal(got, want)
    more = flat.as_strided((2, k), (2 * ld, 1))
    ml.mlora_w4_gather_gemv(route, more, got[:2])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[2])
    del flat, far, more
    torch.cuda.empty_cache()
