"""GPU tests of the products with 4-bit expert weights against fp64.

Tolerance. Weights enter exactly, products are exact (fp32 rows as three bf16
parts), so what is off is fp32 sums. A group's sum runs over values of up to
31 with 16 + zero <= 31 times the sum of x taken off, so its partial sums stay
below 62 sum |x| |s|; with M = sum over k of 62 |x| |s| and at most 4 K roundings
(three parts and the sum of x), the probabilistic bound of tests/common.py
gives 10 sqrt(4 K) u M per element. The relative L2 of an fp32 output: a
rounding is uniform (u / sqrt(3) of a partial sum), 384 of them per group of
128 on partial sums of at most 40 sqrt(128) |x| rms against a result of
4.6 sqrt(128) |x|: below 100 u, less for the smaller groups.  A bf16 output
adds one rounding of 2^-8 per element.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import moe
from tests.common import REL_L2_TOL, rel_l2

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(scope="module")
def ml():
    import moe_expert_lora_amd
    return moe_expert_lora_amd


class Weights:
    def __init__(self, ml, E, K, N, group, zeros, dtype, seed):
        rng = np.random.default_rng(seed)
        self.E, self.K, self.N, self.group, self.dtype = E, K, N, group, DT[dtype]
        self.q = rng.integers(0, 256, size=(E, N, K // 2), dtype=np.uint8)
        shape = (E, N, -(-K // group))
        scales = torch.from_numpy((rng.random(shape) + 0.5) * 0.25 / np.sqrt(K)).to(self.dtype)
        self.zeros = rng.integers(0, 16, size=shape, dtype=np.uint8) if zeros else None
        self.scales = scales.double().numpy()
        self.w = moe.w4_weights(self.q, self.scales, self.zeros, K, group)
        self.route = ml.make_w4_route(
            torch.from_numpy(self.q).to(DEV), scales.to(DEV),
            None if self.zeros is None else torch.from_numpy(self.zeros).to(DEV), K, group)

    def check(self, got, x, ids, top_k, x_by_row, label=""):
        n = got.shape[0]
        host = x.detach().double().cpu().numpy()
        ref = moe.w4_products(self.w, host, ids, top_k, x_by_row, n)
        span = np.abs(self.scales)[..., np.arange(self.K) // self.group] * 62
        mag = moe.w4_products(span, np.abs(host), ids, top_k, x_by_row, n)
        tol = 10 * np.sqrt(4 * self.K) * U * mag
        half = 2.0 ** -8 if self.dtype == torch.bfloat16 else 0.0
        g = got.detach().double().cpu().numpy()
        assert np.isfinite(g).all()
        err = np.abs(g - ref)
        assert (err <= tol + half * (np.abs(ref) + tol)).all(), (label, err.max())
        rel = rel_l2(g, ref)
        print(f"{label}: rel_l2={rel:.3e}", flush=True)
        assert rel <= (REL_L2_TOL if half else 100 * U), label
        if ids is not None:
            dead = (np.asarray(ids) < 0) | (np.asarray(ids) >= self.E)
            assert (g[dead] == 0).all()


def _x(shape, dtype, seed, mean=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) + mean).to(DT[dtype])


def _run(ml, w, x, n, ids, top_k, x_by_row):
    out = torch.full((n, w.N), 9.0, dtype=w.dtype, device=DEV)
    d = None if ids is None else torch.from_numpy(ids).to(DEV)
    ml.mlora_w4_gather_gemv(w.route, x, out, d, top_k, x_by_row=x_by_row)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128, 256, 384])
@pytest.mark.parametrize("rows,k,n", [(1, 128, 64), (1, 1000, 77), (3, 8, 1), (16, 136, 100),
                                      (17, 264, 16), (63, 520, 129), (5, 4088, 33)])
def test_one_weight(ml, dtype, zeros, group, rows, k, n):
    w = Weights(ml, 1, k, n, group, zeros, dtype, rows + k)
    x = _x((rows, k), dtype, 1)
    w.check(_run(ml, w, x, rows, None, 1, False), x, None, 1, False, f"{rows}x{k}x{n}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("x_by_row", [False, True])
@pytest.mark.parametrize("rows,experts,top_k,k,n,group,zeros", [
    (8, 4, 2, 256, 96, 64, True), (40, 16, 8, 768, 512, 128, False),
    (37, 5, 1, 1000, 1365, 32, True), (640, 128, 8, 96, 130, 32, False),
    (300, 2, 1, 328, 65, 128, True), (2100, 3, 2, 64, 24, 64, False),
    (4500, 300, 4, 136, 20, 256, True), (64, 40, 8, 2048, 260, 128, False)])
def test_expert_rows(ml, dtype, x_by_row, rows, experts, top_k, k, n, group, zeros):
    w = Weights(ml, experts, k, n, group, zeros, dtype, rows)
    rng = np.random.default_rng(rows)
    rows -= rows % top_k
    ids = rng.integers(0, experts, size=rows).astype(np.int32)
    ids[rng.random(rows) < 0.1] = -1
    ids[rng.random(rows) < 0.03] = experts
    x = _x((rows if x_by_row else rows // top_k, k), dtype, 2)
    w.check(_run(ml, w, x, rows, ids, top_k, x_by_row), x, ids, top_k, x_by_row,
            f"{rows}/{experts}")


# rows, experts, top_k, k, n, group, zeros: enough column tiles for the form
# that streams them, with one and two row blocks per pass, k in one panel of
# LDS and in several, short last chunks, odd widths, rows past one scan
STREAMED = [(640, 128, 8, 264, 260, 64, True), (640, 128, 8, 136, 289, 128, False),
            (1600, 100, 4, 72, 340, 32, True), (2600, 128, 1, 320, 257, 32, False),
            (4500, 90, 2, 1000, 400, 256, True), (300, 20, 1, 2600, 1700, 128, True),
            (34, 1, 1, 200, 33001, 64, False), (700, 8, 1, 96, 4100, 128, True)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("x_by_row", [False, True])
@pytest.mark.parametrize("rows,experts,top_k,k,n,group,zeros", STREAMED)
def test_streamed_expert_rows(ml, dtype, x_by_row, rows, experts, top_k, k, n, group, zeros):
    w = Weights(ml, experts, k, n, group, zeros, dtype, rows)
    rng = np.random.default_rng(rows)
    ids = None
    if experts > 1:
        ids = rng.integers(0, experts, size=rows).astype(np.int32)
        ids[rng.random(rows) < 0.1] = -1
        ids[rng.random(rows) < 0.03] = experts
        ids[rows // 2:rows // 2 + 40] = 1       # one expert with more rows than a pass
    x = _x((rows if x_by_row else -(-rows // top_k), k), dtype, 2)
    w.check(_run(ml, w, x, rows, ids, top_k, x_by_row), x, ids, top_k, x_by_row,
            f"{rows}/{experts}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,experts,k,n,group,zeros", [
    (1, 16, 264, 100, 32, True), (8, 52, 1080, 314, 64, False), (15, 16, 2048, 100, 128, True),
    (20, 64, 1000, 1000, 32, True), (9, 40, 2104, 1900, 128, False)])
def test_fewer_rows_than_experts(ml, dtype, rows, experts, k, n, group, zeros):
    """Places are rows: repeated experts, rows without one, all the same."""
    w = Weights(ml, experts, k, n, group, zeros, dtype, rows)
    x = _x((rows, k), dtype, 9)
    rng = np.random.default_rng(rows)
    mixed = rng.integers(0, experts, size=rows).astype(np.int32)
    mixed[rows // 2:] = mixed[0]
    mixed[rows // 3] = -1
    mixed[-1] = experts + 3
    for ids in (mixed, np.full(rows, experts - 1, np.int32), np.full(rows, -1, np.int32),
                np.arange(rows, dtype=np.int32)):
        w.check(_run(ml, w, x, rows, ids, 1, True), x, ids, 1, True, f"{rows}/{experts}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,experts,k,n,group,zeros", [
    (5, 4, 2104, 4000, 64, True),      # four waves to a pair, several panels in float32
    (90, 4, 2504, 4010, 128, False),   # two row blocks, several panels
    (40, 16, 704, 1200, 32, True),
    (60, 16, 1200, 1030, 64, True),    # three waves to a pair
    (70, 32, 1000, 1000, 128, False)])  # two, the last tile alone in its pair
def test_several_waves_to_a_pair(ml, dtype, rows, experts, k, n, group, zeros):
    w = Weights(ml, experts, k, n, group, zeros, dtype, rows)
    x = _x((rows, k), dtype, 10)
    ids = np.random.default_rng(rows).integers(-1, experts, size=rows).astype(np.int32)
    w.check(_run(ml, w, x, rows, ids, 1, True), x, ids, 1, True, f"{rows}/{experts}")


def test_streamed_non_finite_rows_stay_alone(ml):
    w = Weights(ml, 64, 200, 520, 64, True, "bf16", 17)
    x = _x((300, 200), "bf16", 5)
    ids = (np.arange(300) % 64).astype(np.int32)
    clean = _run(ml, w, x, 300, ids, 1, False)
    x[4, 10] = float("inf")
    x[9, 199] = float("nan")
    got = _run(ml, w, x, 300, ids, 1, False)
    keep = [r for r in range(300) if r not in (4, 9)]
    assert torch.equal(got[keep], clean[keep])
    assert not torch.isfinite(got[4]).any() and torch.isnan(got[9]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_sided_routing(ml, dtype):
    w = Weights(ml, 9, 264, 50, 64, True, dtype, 5)
    x = _x((130, 264), dtype, 3)
    for fill in (-1, 0, 8, 9):
        ids = np.full(130, fill, dtype=np.int32)
        w.check(_run(ml, w, x, 130, ids, 1, False), x, ids, 1, False, f"all {fill}")


@pytest.mark.parametrize("zeros", [False, True])
def test_rows_with_a_mean(ml, zeros):
    """Rows whose values do not average out: the offset's share is large."""
    w = Weights(ml, 1, 1024, 200, 128, zeros, "bf16", 6)
    x = _x((20, 1024), "bf16", 4, mean=3.0)
    w.check(_run(ml, w, x, 20, None, 1, False), x, None, 1, False, "mean 3")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_non_finite_rows_stay_alone(ml, dtype):
    w = Weights(ml, 3, 256, 100, 128, False, dtype, 7)
    x = _x((40, 256), dtype, 5)
    ids = (np.arange(40) % 3).astype(np.int32)
    clean = _run(ml, w, x, 40, ids, 1, False)
    x[4, 10] = float("inf")
    x[9, 255] = float("nan")
    ids[11] = -1
    x[11] = float("nan")                              # a skipped row's x is not used
    got = _run(ml, w, x, 40, ids, 1, False)
    keep = [r for r in range(40) if r not in (4, 9, 11)]
    assert torch.equal(got[keep], clean[keep])
    assert not torch.isfinite(got[4]).any() and torch.isnan(got[9]).all()
    assert bool((got[11] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides(ml, dtype):
    w = Weights(ml, 4, 200, 60, 32, True, dtype, 8)
    x = _x((24, 200), dtype, 6)
    ids = np.random.default_rng(8).integers(-1, 4, size=48).astype(np.int32)
    want = _run(ml, w, x, 48, ids, 2, False)
    wide = torch.full((24, 264), float("nan"), dtype=x.dtype, device=DEV)
    wide[:, 16:216] = x
    for lead, ld in ((0, 60), (4, 72), (1, 63)):
        buf = torch.full((48, ld + lead), 5.0, dtype=x.dtype, device=DEV)
        view = buf[:, lead:lead + 60]
        ml.mlora_w4_gather_gemv(w.route, wide[:, 16:216], view, torch.from_numpy(ids).to(DEV), 2)
        assert torch.equal(view, want)
        assert bool((buf[:, :lead] == 5).all()) and bool((buf[:, lead + 60:] == 5).all())


def test_output_rows_past_32_bit_offsets(ml):
    w = Weights(ml, 1, 64, 32, 32, False, "bf16", 9)
    x = _x((3, 64), "bf16", 7)
    want = _run(ml, w, x, 3, None, 1, False)
    ld = (1 << 31) + 64
    flat = torch.empty(2 * ld + 64, dtype=torch.bfloat16, device=DEV)
    view = flat.as_strided((3, 32), (ld, 1))
    ml.mlora_w4_gather_gemv(w.route, x, view)
    torch.cuda.synchronize()
    assert torch.equal(view, want)


def test_graph_replay(ml):
    """Captured once; each replay, after ids and x were rewritten, equals the
    eager call bit for bit."""
    w = Weights(ml, 16, 384, 250, 64, True, "bf16", 10)
    ids = torch.zeros(64, dtype=torch.int32, device=DEV)
    x = torch.zeros((16, 384), dtype=torch.bfloat16, device=DEV)
    out = torch.zeros((64, 250), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            ml.mlora_w4_gather_gemv(w.route, x, out, ids, 4)
    torch.cuda.current_stream().wait_stream(side)
    for r in range(4):
        host = np.random.default_rng(r).integers(-1, 16, size=64).astype(np.int32)
        ids.copy_(torch.from_numpy(host))
        x.copy_(_x((16, 384), "bf16", 20 + r))
        eager = _run(ml, w, x, 64, host, 4, False)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), r
        w.check(out, x, host, 4, False, f"replay {r}")


def test_binding_refuses(ml):
    w = Weights(ml, 2, 64, 32, 32, False, "bf16", 11)
    x = _x((4, 64), "bf16", 8)
    out = torch.empty((4, 32), dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros(4, dtype=torch.int32, device=DEV)
    q, s = torch.from_numpy(w.q).to(DEV), torch.ones((2, 32, 2), device=DEV)
    for call in (
            lambda: ml.mlora_w4_gather_gemv(w.route, x[:, :56], out, ids),
            lambda: ml.mlora_w4_gather_gemv(w.route, x, out, ids[:3]),
            lambda: ml.mlora_w4_gather_gemv(w.route, x, out[:, :16], ids),
            lambda: ml.mlora_w4_gather_gemv(w.route, x.cpu(), out, ids),
            lambda: ml.make_w4_route(q, s, None, 128, 32),
            lambda: ml.make_w4_route(q, s, None, 64, 64),
            lambda: ml.make_w4_route(q, s, q, 64, 32)):
        with pytest.raises(ValueError):
            call()
    for call in (
            lambda: ml.mlora_w4_gather_gemv(w.route, x.float(), out, ids),
            lambda: ml.mlora_w4_gather_gemv(w.route, x, out, ids.long()),
            lambda: ml.make_w4_route(q.char(), s, None, 64, 32),
            lambda: ml.make_w4_route(q, s.half(), None, 64, 32)):
        with pytest.raises(TypeError):
            call()
    for call in (
            lambda: ml.mlora_w4_gather_gemv(w.route, x, out),          # two experts, no ids
            lambda: ml.mlora_w4_gather_gemv(w.route, x, out, ids, 0),
            lambda: ml.make_w4_route(q, torch.ones((2, 32, 4), device=DEV), None, 64, 16)):
        with pytest.raises(ml.MloraError):
            call()
