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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_activated_rows_keep_24_bits(ml, dtype):
    """Two hidden columns whose activations differ in their 17th bit or so cancel in the
    last product, so that what is left shows their last bits.

    x has two values, gate's rows are alike and up's differ in one small code, so every
    value before the last product is a handful of roundings: up one sum and its scale,
    silu(gate) shared, times up and p; then three parts of each column and the scale.
    Column by column (4 + 3 + 1) roundings, 6 shared ones: 16 times 2^-24 of the two
    columns' magnitudes covers them. Rows of 18 bits are off by up to 64."""
    dim, hidden, T, E = 128, 2, 16, 24
    rng = np.random.default_rng(3)
    code = lambda v: fp8.e4m3_round(np.asarray(v, dtype=np.float64))  # noqa: E731
    gate, up, down = np.zeros((E, 2, dim)), np.zeros((E, 2, dim)), np.zeros((E, dim, 2))
    gate[:, :, :2] = rng.uniform(100, 400, (E, 1, 2))
    up[:, :, 0] = rng.uniform(300, 448, (E, 1))
    up[:, 1, 1] = rng.uniform(0.25, 2, E)
    down[:, :, 0] = rng.uniform(100, 448, (E, dim))
    down[:, :, 1] = -down[:, :, 0]
    made = [(code(w), rng.uniform(0.002, 0.004, (E, 1, 1)).astype(np.float32))
            for w in (gate, up, down)]
    for seed in range(8):
        c = Case(ml, seed, T, E, 1, dim, hidden, dtype)
        c.routes = [ml.make_fp8_route(dev(w), dev(s)) for w, s in made]
        c.full = [fp8.expand(w, s) for w, s in made]
        c.x.zero_()
        c.x[:, 0] = dev(rng.uniform(1, 2, T)).to(c.x.dtype)
        c.x[:, 1] = dev(rng.uniform(1, 2, T) * 2.0 ** -8).to(c.x.dtype)
        c.run(renorm=False)
        x = to64(c.x)
        ref, idx, w, _ = fp8.layer(x, to64(c.logits), *c.full, 1, False)
        mag = np.zeros_like(ref)
        for t in range(T):
            g, u, d = (m[idx[t, 0]] for m in c.full)
            mag[t] = np.abs(d) @ np.abs(w[t, 0] * fp8.silu(g @ x[t]) * (u @ x[t]))
        # the weights are the kernel's own: a few units of the exponential
        close(to64(c.w), w, w * 64 * F32)
        ref, mag = ref * to64(c.w) / w, mag * to64(c.w) / w
        err = mag * 16 * F32
        close(to64(c.out), ref, err + (np.abs(ref) + err) * U[dtype])
