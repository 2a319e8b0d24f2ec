"""GPU tests of every form of the MoE layer's first kernel (by the 128-blocks of a row of
x and the waves that share them), whole and ragged, and of the ends of x's range."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8  # noqa: E402
from tests.fp8_cases import F32, U, close, to64  # noqa: E402
from tests.test_gpu_few_tokens import Case, dev  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def ml():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_lora_amd
    return moe_expert_lora_amd


# blocks of x: 1, 2, up to 4, up to 8 (one a wave), up to 16 (two), up to 32 (four of bf16;
# fp32 reads them again from here on), more. Whole rows, short last blocks, and numbers of
# blocks that waves share unevenly.
DIMS = [128, 77, 256, 200, 384, 512, 450, 640, 1024, 900, 1100, 1930, 2048, 2100, 3000, 3584, 4096,
        4224, 5000, 7168]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 16])
@pytest.mark.parametrize("dim", DIMS)
def test_form(ml, dim, T, dtype):
    Case(ml, dim + T, T, 6, 3, dim, 136, dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [128, 1100, 2048, 4500])
def test_largest_x(ml, dim, dtype):
    """x of 2^112 and of one sign against codes of 448: a block's sum of products is 2^112
    * 448 * 128 = 2^127.8 before its scale, of 2^-127 over the blocks here, brings gate
    and up down to 1.75. Every value is a power of two or 1.75 of one and the sums are
    exact, so the result is off by silu's few roundings and its parts."""
    T, E, k, hidden = 3, 4, 2, 72
    c = Case(ml, 1, T, E, k, dim, hidden, dtype)
    blocks = -(-dim // 128)
    code = int(fp8.e4m3_round(np.array([448.0]))[0])
    made = []
    for n, m, scale in ((hidden, dim, 2.0 ** -127), (hidden, dim, 2.0 ** -127),
                        (dim, hidden, 2.0 ** -10)):
        w = np.full((E, n, m), code, dtype=np.uint8)
        made.append((w, np.full((E, -(-n // 128), -(-m // 128)), scale / (blocks if m == dim else 1),
                                dtype=np.float32)))
    c.routes = [ml.make_fp8_route(dev(w), dev(s)) for w, s in made]
    c.full = [fp8.expand(w, s) for w, s in made]
    c.x.fill_(2.0 ** 112)
    c.x[1].neg_()
    c.run()
    ref, _, _, _ = fp8.layer(to64(c.x), to64(c.logits), *c.full, k, True)
    assert np.isfinite(ref).all() and (np.abs(ref) > 1e-3).all()
    # scales below 2^-126 are whole multiples of 2^-149 all the same: 1 / blocks of 2^-127
    # rounds to 2^-22 of itself at least, in c.full as in the kernel
    err = np.abs(ref) * ((hidden + 64) * F32 + 2.0 ** -16)
    close(to64(c.out), ref, err + (np.abs(ref) + err) * U[dtype])


@pytest.mark.parametrize("e", [-100, -112])
@pytest.mark.parametrize("dim", [128, 1100, 4500])
def test_smallest_x(ml, dim, e):
    """float32 values of x enter to within 2^-126 (what matrix instructions may take as
    0 of a value's parts)."""
    c = Case(ml, 2, 5, 6, 2, dim, 72, "f32")
    rng = np.random.default_rng(dim)
    made = []
    for n, m in ((72, dim), (72, dim), (dim, 72)):
        w = fp8.e4m3_round(rng.normal(0, 110, (6, n, m)).clip(-448, 448))
        s = rng.uniform(0.5, 2, (6, -(-n // 128), -(-m // 128))) / (40 * np.sqrt(m))
        made.append((w, (s * (2.0 ** -e if m == dim else 1)).astype(np.float32)))
    c.routes = [ml.make_fp8_route(dev(w), dev(s)) for w, s in made]
    c.full = [fp8.expand(w, s) for w, s in made]
    c.x.copy_(dev(rng.normal(0, 1, (5, dim)) * 2.0 ** e))
    c.run()
    x = to64(c.x)
    ref, idx, wts, mag = fp8.layer(x, to64(c.logits), *c.full, 2, True)
    # as mag, of x's own 2^-126
    lost = np.zeros_like(ref)
    for t in range(5):
        for j in range(2):
            g, u, d = (m[idx[t, j]] for m in c.full)
            ge, ue = np.abs(g).sum(1) * 2.0 ** -126, np.abs(u).sum(1) * 2.0 ** -126
            lost[t] += wts[t, j] * (np.abs(d) @ (1.1 * ge * np.abs(u @ x[t])
                                                 + np.abs(fp8.silu(g @ x[t])) * ue + 2 * ge * ue))
    err = mag * (dim + 72 + 96 + 1) * F32 + lost
    close(to64(c.out), ref, err + (np.abs(ref) + err) * U["f32"])
