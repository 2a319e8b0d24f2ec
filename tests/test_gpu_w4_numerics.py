"""GPU tests of how exact the products with 4-bit weights are in fp32, where
x has a mean and the values of a group do not average out.

Tolerance. A group of at most 128 values starts from (z - 7.5) times its sum of
x and adds its products with v - 7.5, whose rms over the 16 values of v is
sqrt(255 / 12) = 4.61. A partial sum is then at most
D + W, D = |z - 7.5| |sum x|, W = 4.61 |x|, the last the size of the sum of
products (the walk's end, its largest). Three parts of x make 3 x 128 additions,
each off by a rounding that is uniform in half a step (rms u / sqrt(3) of the
partial sum), so a group is off by sqrt(384 / 3) u (D + W) |s|, and a row by the
root of the groups' squares; the sum over groups adds a rounding of a result's
size for each of them. No headroom is added: the additions are not all rounded
at the largest partial sum.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import moe
from tests.common import rel_l2

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


def _weights(ml, E, K, N, group, zeros, dtype, seed):
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 256, size=(E, N, K // 2), dtype=np.uint8)
    shape = (E, N, -(-K // group))
    s = torch.from_numpy((rng.random(shape) + 0.5) * 0.25 / np.sqrt(K)).to(dtype)
    z = rng.integers(0, 16, size=shape, dtype=np.uint8) if zeros else None
    route = ml.make_w4_route(torch.from_numpy(q).to(DEV), s.to(DEV),
                             None if z is None else torch.from_numpy(z).to(DEV), K, group)
    return route, q, s.double().numpy(), z


def _bound(x, s, z, K, group, ref):
    """rms error of the rows of one expert, by the formula above."""
    var = np.zeros_like(ref)
    per = min(group, 128)
    for k0 in range(0, K, per):
        xs = x[:, k0:k0 + per]
        g = k0 // group
        zero = 8.0 if z is None else z[:, g].astype(float)
        d = np.abs(zero - 7.5) * np.abs(xs.sum(1))[:, None]
        w = np.sqrt(255 / 12) * np.sqrt((xs ** 2).sum(1))[:, None]
        var += (384 / 3) * (U * (d + w) * np.abs(s[:, g])[None, :]) ** 2
        var += (U * ref) ** 2 / 3
    return np.sqrt(var)


MAKE = {"mean 0": lambda r, sh: r.normal(size=sh), "mean 3": lambda r, sh: r.normal(size=sh) + 3,
        "squared relu": lambda r, sh: np.maximum(r.normal(size=sh), 0) ** 2}


@pytest.mark.parametrize("values", list(MAKE))
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("experts,rows,k,n,group", [
    (1, 20, 768, 200, 128), (1, 20, 768, 200, 32), (1, 9, 1000, 77, 64), (1, 3, 1280, 64, 384),
    (64, 130, 264, 520, 64), (64, 200, 520, 290, 128)])
def test_float32_rows_with_a_mean(ml, values, zeros, experts, rows, k, n, group):
    route, q, s, z = _weights(ml, experts, k, n, group, zeros, torch.float32, k + rows)
    host = MAKE[values](np.random.default_rng(rows), (rows, k)).astype(np.float32)
    ids = None if experts == 1 else (np.arange(rows) % experts).astype(np.int32)
    out = torch.empty((rows, n), device=DEV)
    ml.mlora_w4_gather_gemv(route, torch.from_numpy(host).to(DEV), out,
                            None if ids is None else torch.from_numpy(ids).to(DEV))
    got, x = out.double().cpu().numpy(), host.astype(np.float64)
    w = moe.w4_weights(q, s, z, k, group)
    ref = moe.w4_products(w, x, ids, 1, True, rows)
    lim = np.empty_like(ref)
    for r in range(rows):
        e = 0 if ids is None else ids[r]
        lim[r] = _bound(x[r:r + 1], s[e], None if z is None else z[e], k, group, ref[r:r + 1])[0]
    rel, tol = rel_l2(got, ref), np.linalg.norm(lim) / np.linalg.norm(ref)
    print(f"{values} {experts}x{k}x{n} g{group}: rel_l2 {rel / U:.2f} u, limit {tol / U:.2f} u",
          flush=True)
    assert rel <= tol


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_every_weight_is_exact(ml, zeros, group):
    """x rows of the identity read the weights out: v - z times the scale,
    rounded once, in every place of the packed words."""
    k, n = 264, 130
    route, q, s, z = _weights(ml, 1, k, n, group, zeros, torch.float32, 5)
    out = torch.empty((k, n), device=DEV)
    ml.mlora_w4_gather_gemv(route, torch.eye(k, device=DEV), out)
    want = moe.w4_weights(q, s, z, k, group)[0].T
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= U * np.abs(want)).all()


def _one_row_each(ml, dtype, zeros, group, special):
    """Rows of ordinary values with ``special`` in row 3, and the same without it."""
    k, n, rows = 264, 520, 40
    route, q, s, z = _weights(ml, 2, k, n, group, zeros, dtype, 9)
    x = torch.randn((rows, k), generator=torch.Generator(device=DEV).manual_seed(6),
                    device=DEV).to(dtype)
    ids = (torch.arange(rows, device=DEV) % 2).to(torch.int32)
    clean, got = (torch.empty((rows, n), dtype=dtype, device=DEV) for _ in range(2))
    ml.mlora_w4_gather_gemv(route, x, clean, ids)
    x[3] = special.to(DEV)
    ml.mlora_w4_gather_gemv(route, x, got, ids)
    keep = [r for r in range(rows) if r != 3]
    assert torch.equal(got[keep], clean[keep])
    w = moe.w4_weights(q, s, z, k, group)[1]
    scale = s[1][:, np.arange(k) // group]
    return w, scale, x[3].double().cpu().numpy(), got[3].double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("signs", ["same", "mixed"])
def test_largest_values(ml, dtype, zeros, group, signs):
    """A whole row of 2^117, the largest that the header names: finite and right
    (scales below 2^-4 keep the sums over groups in range). Its neighbours stay
    as they are. A group's 128 sums and its start are each off by half a step of
    at most 15 sum |x|; the scaled sum over groups by one of its own size."""
    big = torch.full((264,), 2.0 ** 117)
    if signs == "mixed":
        big[::3] = -big[::3]
    w, scale, x, got = _one_row_each(ml, dtype, zeros, group, big.to(dtype))
    ref = w @ x
    tol = (3 * 129 + 264) * U * 15 * (np.abs(scale) @ np.abs(x))
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol + half * (np.abs(ref) + tol)).all()


@pytest.mark.parametrize("dtype,size", [(torch.float32, 2.0 ** -104), (torch.float32, 2.0 ** -112),
                                        (torch.float32, 2.0 ** -124), (torch.float32, 2.0 ** -130),
                                        (torch.bfloat16, 2.0 ** -120),
                                        (torch.bfloat16, 2.0 ** -130)])
def test_smallest_values(ml, dtype, size):
    """Values enter to within 2^-126; a sum that is subnormal may be 0, at each of
    the additions (three parts, a start, one for the groups)."""
    g = torch.Generator().manual_seed(8)
    row = (torch.randn(264, generator=g, dtype=torch.float64) * size).to(dtype)
    w, scale, x, got = _one_row_each(ml, dtype, True, 64, row)
    ref = w @ x
    mag = 15 * (scale @ np.abs(x))
    tol = 2.0 ** -126 * (np.abs(w).sum(1) + 5 * scale.sum(1) + 1) + 1056 * U * mag
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert (np.abs(got - ref) <= tol + half * np.abs(ref)).all()
