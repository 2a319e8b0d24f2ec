"""GPU tests of the 4-bit products in every form of the launch plan
(w4_cases.FORMS; test_w4_plan.py keeps the list whole), against fp64 on the device.

Tolerance. A group's partial sums stay below 15 sum |x| |s| (from (z - 7.5) sum x
to the sum of products with v - 7.5); with at most 4 K roundings (three parts and
the start), the probabilistic bound is 10 sqrt(4 K) u 15 sum |x| |s| per element.
The relative L2 of an fp32 output for x of mean 0: roundings of rms u / sqrt(3),
384 a group of 128, on partial sums of at most (4.61 + 4.61) sqrt(128) |x| rms
(zero points drawn as the values are) against a result of 6.52 sqrt(128) |x|:
16 u, and one for the sums over groups. A bf16 output adds one rounding of 2^-8
per element.
"""
from __future__ import annotations

import pytest

from tests.common import REL_L2_TOL
from tests.w4_cases import FORMS

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ml():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_lora_amd
    return moe_expert_lora_amd


def _ids(g, rows, experts):
    """Uniform, a tenth dropped, some past the experts, a run of 40 of one expert
    (more than a pass) in calls of more rows than that."""
    ids = torch.randint(0, experts, (rows,), generator=g, device=DEV, dtype=torch.int32)
    u = torch.rand(rows, generator=g, device=DEV)
    ids[u < 0.1] = -1
    ids[u > 0.98] = experts
    if rows > 80:
        ids[rows // 3:rows // 3 + 40] = experts - 1
    return ids


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,experts,k,n,group,f32,form", FORMS)
def test_form(ml, rows, experts, k, n, group, f32, form, zeros):
    dtype, E = (torch.float32 if f32 else torch.bfloat16), max(experts, 1)
    g = torch.Generator(device=DEV).manual_seed(rows * 31 + k)
    groups = -(-k // group)
    q = torch.randint(0, 256, (E, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = ((torch.rand((E, n, groups), generator=g, device=DEV) + 0.5) * 0.25 / k ** 0.5).to(dtype)
    z = torch.randint(0, 16, (E, n, groups), generator=g, device=DEV,
                      dtype=torch.uint8) if zeros else None
    route = ml.make_w4_route(q, s, z, k, group)
    top_k = 2 if rows % 2 == 0 else 1
    x = torch.randn((rows // top_k, k), generator=g, device=DEV).to(dtype)
    ids = _ids(g, rows, E) if experts else None
    ld = n + 3 if rows % 3 == 0 else n                    # rows that start anywhere
    buf = torch.full((rows, ld), 9.0, dtype=dtype, device=DEV)
    out = buf[:, :n]
    ml.mlora_w4_gather_gemv(route, x, out, ids, top_k)
    torch.cuda.synchronize()
    assert bool((buf[:, n:] == 9).all())
    err2 = ref2 = 0.0
    src = torch.arange(rows, device=DEV) // top_k
    half = 0.0 if f32 else 2.0 ** -8
    for e in range(E):
        r = torch.arange(rows, device=DEV) if ids is None else torch.nonzero(ids == e).flatten()
        if r.numel() == 0:
            continue
        sc = s[e].double().repeat_interleave(group, 1)[:, :k]
        zero = 8.0 if z is None else z[e].double().repeat_interleave(group, 1)[:, :k]
        w = (torch.stack((q[e] & 15, q[e] >> 4), 2).flatten(1).double() - zero) * sc
        xs = x[src[r]].double()
        ref, mag = xs @ w.t(), xs.abs() @ sc.t()
        got = out[r].double()
        tol = 10 * (4 * k) ** 0.5 * U * 15 * mag
        bad = (got - ref).abs() > tol + half * (ref.abs() + tol)
        assert bool(torch.isfinite(got).all()) and not bool(bad.any()), \
            (e, r[bad.any(1)].tolist()[:4], torch.nonzero(bad)[:4].tolist())
        err2 += float(((got - ref) ** 2).sum())
        ref2 += float((ref ** 2).sum())
    if ref2 > 0:
        rel = (err2 / ref2) ** 0.5
        print(f"{form}: rel_l2={rel:.3e}", flush=True)
        assert rel <= (17 * U if f32 else REL_L2_TOL)
    if ids is not None:
        assert not bool(out[(ids < 0) | (ids >= E)].any())
