"""GPU tests of the 8-bit products: the rows' quantiser (codes against the
definition), the packed weights and the product over rows sorted by expert."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8, moe  # noqa: E402
from tests.fp8_cases import F32, U, close, product_error, to64, weights  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ml():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_lora_amd
    return moe_expert_lora_amd


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def strided(t, extra):
    """The same values in rows that lie ``extra`` elements further apart, behind
    one element that moves their start."""
    wide = torch.zeros((t.shape[0], t.shape[1] + extra), dtype=t.dtype, device=DEV)
    view = wide[:, 1:1 + t.shape[1]] if extra else wide
    view.copy_(t)
    return view


def quantised(ml, x, up=None, q=None):
    k = x.shape[1]
    if q is None:
        q = torch.full((x.shape[0], ml.mlora_fp8_row_width(k)), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((-(-k // 128), x.shape[0]), 7.0, device=DEV)
    ml.mlora_fp8_quant(x, q, s, up=up)
    assert (q[:, whole(k):] == 0x55).all()  # a block that only moves the next row
    return q, s


def whole(k):
    return -(-k // 128) * 128


def rows_in(ml, codes):
    """Quantised rows as the product takes them; the block behind them holds NaN."""
    t = torch.full((codes.shape[0], ml.mlora_fp8_row_width(codes.shape[1])), 0x7f,
                   dtype=torch.uint8, device=DEV)
    t[:, :codes.shape[1]] = dev(codes)
    return t


# -- quantiser ---------------------------------------------------------------

QUANT = [(1, 1), (1, 128), (3, 127), (5, 129), (64, 768), (7, 2048), (33, 1000), (2, 4100)]


@pytest.mark.parametrize("extra", [0, 8, 3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k", QUANT)
def test_quant(ml, rows, k, dtype, extra):
    rng = np.random.default_rng(rows * 31 + k)
    x = dev(rng.normal(0, 1, (rows, k)) * 2.0 ** rng.integers(-20, 20, (rows, 1))).to(TORCH[dtype])
    q, s = quantised(ml, strided(x, extra))
    codes, scales = fp8.quantise(to64(x), whole(k))
    got = q[:, :whole(k)].cpu().numpy()
    # codes of a zero keep its sign; both are 0
    assert np.array_equal(fp8.e4m3_decode(got), fp8.e4m3_decode(codes))
    assert not got[:, k:].any()
    close(to64(s), scales, np.abs(scales) * F32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quant_ties_and_neighbours(ml, dtype):
    """Values half way between two codes, and fp32's neighbours of them, for
    largest values whose quotients do not come out even."""
    table = fp8.e4m3_values()
    mid = ((table[1:] + table[:-1]) / 2)[:120]
    for top in (448.0, 1.0, 1.5, 3.0, 7.0, 5.0, 0.328125, 1.9921875):
        v = np.zeros((6, 128))
        v[:, 127] = top
        exact = torch.from_numpy(mid * top / 448).to(TORCH[dtype])
        near = exact.float().numpy()
        for i, w in enumerate((near, -near, np.nextafter(near, np.float32(1e9)),
                               np.nextafter(near, np.float32(0)), near * 1.001, near * 0.999)):
            v[i, :mid.size] = w
        x = dev(v.astype(np.float32)).to(TORCH[dtype])
        codes, _ = fp8.quantise(to64(x), 128)
        q, _ = quantised(ml, x)
        assert np.array_equal(fp8.e4m3_decode(q.cpu().numpy()), fp8.e4m3_decode(codes)), top


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quant_extremes(ml, dtype):
    """Zeros, subnormals, the largest values, infinities and NaN: a group of its own
    each; groups beside a non-finite one keep their values."""
    big = float(torch.finfo(TORCH[dtype]).max)
    tiny = 2.0 ** -133
    rows = [[0.0] * 3, [tiny, -tiny, 0], [2.0 ** -126, tiny, 1e-30], [big, -big / 3, 1.0],
            [big, 2.0 ** -100, -big], [np.inf, 1, 2], [1, -np.inf, 2], [np.nan, 1, 2],
            [np.inf, np.nan, -np.inf], [1.75 * 2.0 ** -118, 2.0 ** -124, -2.0 ** -122]]
    v = np.zeros((len(rows), 256), dtype=np.float32)
    v[:, :3] = rows
    v[:, 200] = 3.0
    x = dev(v).to(TORCH[dtype])
    codes, scales = fp8.quantise(to64(x), 256)
    q, s = quantised(ml, x)
    assert np.array_equal(fp8.e4m3_decode(q[:, :256].cpu().numpy()), fp8.e4m3_decode(codes))
    close(to64(s), scales, np.abs(scales) * F32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,extra", [(1, 40, 0), (9, 768, 0), (4, 1001, 5), (70, 256, 8)])
def test_quant_silu(ml, rows, k, extra, dtype):
    """silu(x) up within its fp32 evaluation (8 roundings) of half a code."""
    rng = np.random.default_rng(k)
    gate, up = (dev(rng.normal(0, 3, (rows, k))).to(TORCH[dtype]) for _ in range(2))
    gate[0, 0], gate[-1, k - 1] = -200.0, 200.0
    both = torch.cat([strided(gate, extra), strided(up, extra)], 1) if extra == 0 else None
    g, u = (both[:, :k], both[:, k:]) if both is not None else (strided(gate, extra),
                                                               strided(up, extra))
    q, s = quantised(ml, g, u)
    want = fp8.silu(to64(gate)) * to64(up)
    got = fp8.rows_of(q.cpu().numpy(), s.cpu().numpy(), k)
    scale = to64(s).T[:, np.arange(k) // 128]
    close(got, want, np.maximum(np.abs(want) * 2.0 ** -4, scale * 2.0 ** -10) * (1 + 2.0 ** -10)
          + np.abs(want) * 10 * F32)
    top = np.abs(np.pad(want, ((0, 0), (0, -k % 128)))).reshape(rows, -1, 128).max(2)
    close(to64(s).T, np.maximum(top, 448 * 2.0 ** -126) / 448, top / 448 * 10 * F32)


def test_quant_leaves_the_rest(ml):
    """Rows and columns outside the call keep their bytes."""
    x = torch.randn((5, 100), device=DEV)
    wide = torch.full((7, 160), 0x33, dtype=torch.uint8, device=DEV)
    ml.mlora_fp8_quant(x, wide[1:6, 16:144], torch.empty((1, 5), device=DEV))
    rest = wide.cpu().numpy().copy()
    rest[1:6, 16:144] = 0x33
    assert (rest == 0x33).all()


# -- product -----------------------------------------------------------------

def spans(rng, n, E, lead=0, behind=0, skew=False):
    """Offsets of E spans over n rows: the first ``lead`` and last ``behind`` rows are
    in none."""
    p = rng.dirichlet(np.full(E, 0.3 if skew else 5.0))
    counts = rng.multinomial(n - lead - behind, p)
    if E > 2:
        counts[1] += counts[2]
        counts[2] = 0
    return np.concatenate([[lead], lead + counts.cumsum()]).astype(np.int32)


def check_product(ml, seed, E, N, K, n, dtype, ids=False, top_k=1, lead=0, behind=0, skew=False,
                  one=False, transpose=False, out_extra=0):
    rng = np.random.default_rng(seed)
    w, ws = weights(rng, E, K, N) if transpose else weights(rng, E, N, K)
    q_rows = n // top_k if ids else n
    codes, qs = fp8.quantise(rng.normal(0, 1, (q_rows, K)), whole(K))
    qs = qs.astype(np.float32)
    off = None if one else spans(rng, n, E, lead, behind, skew)
    order = None
    if ids:
        order = rng.permutation(n).astype(np.int32)
        order[::17] = -1
        order[5::29] = q_rows * top_k + 3
    base = rng.normal(0, 1, (n, N)).astype(np.float32)
    out = strided(dev(base).to(TORCH[dtype]), out_extra)
    before = to64(out)
    route = ml.make_fp8_route(dev(w).view(torch.float8_e4m3fn), dev(ws), transpose=transpose)
    ml.mlora_fp8_gemm(route, rows_in(ml, codes), dev(qs), out, None if off is None else dev(off),
                      None if order is None else dev(order), top_k)
    full = fp8.expand(w, ws)
    if transpose:
        full = full.transpose(0, 2, 1)
    ref, mag = fp8.products(full, fp8.rows_of(codes, qs, K), off, order, top_k, before)
    close(to64(out), ref, np.where(mag > 0, product_error(ref, mag, K, dtype), 0.0))


# E, N, K, rows: one value, ragged, more experts than rows, few long spans; then each
# of the larger tiles (64 x 128, 128 x 128, 256 x 256), odd numbers of blocks
LARGE = [(40, 260, 384, 1300), (5, 3900, 130, 1500), (3, 4000, 300, 2100), (9, 4100, 129, 3600),
         (2, 2300, 640, 8300)]
SIZES = [(1, 1, 1, 1), (3, 5, 7, 11), (4, 100, 300, 37), (16, 130, 129, 5), (5, 365, 1000, 203),
         (128, 64, 256, 640), (2, 257, 640, 700), (1, 2048, 2048, 1), (3, 16, 2100, 60),
         (1000, 33, 128, 300), (2, 1030, 130, 1500)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,N,K,n", SIZES)
def test_product(ml, E, N, K, n, dtype):
    check_product(ml, N + K, E, N, K, n, dtype, skew=n % 2 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("skew", [False, True])
@pytest.mark.parametrize("E,N,K,n", LARGE)
def test_product_in_large_tiles(ml, E, N, K, n, skew, dtype):
    check_product(ml, N + K, E, N, K, n, dtype, skew=skew, ids=skew, lead=3 * skew, behind=5 * skew)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,n", [(1, 1, 1), (48, 4000, 3), (300, 512, 16), (129, 257, 17),
                                   (256, 384, 300), (1000, 200, 1025), (4097, 257, 8200),
                                   (4000, 128, 2050)])
def test_product_of_one_weight(ml, N, K, n, dtype):
    check_product(ml, n, 1, N, K, n, dtype, one=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,N,K,n,top_k", [(8, 100, 300, 64, 4), (128, 70, 256, 640, 8),
                                           (3, 260, 130, 1200, 2), (6, 30, 90, 6, 6)])
def test_product_of_token_rows(ml, E, N, K, n, top_k, dtype):
    """Through sorted ids, some of them -1 or past the tokens; rows in front of and
    behind the spans stay as they were."""
    check_product(ml, n + E, E, N, K, n, dtype, ids=True, top_k=top_k)
    check_product(ml, n + E, E, N, K, n, dtype, ids=True, top_k=top_k, lead=3, behind=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,N,K,n", [(1, 7, 3, 2), (4, 300, 100, 37), (2, 640, 257, 600)])
def test_product_of_transposed_weights(ml, E, N, K, n, dtype):
    check_product(ml, n, E, N, K, n, dtype, transpose=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("extra", [1, 4, 7])
@pytest.mark.parametrize("N,n", [(101, 30), (101, 900), (4061, 4500)])
def test_product_into_wider_rows(ml, extra, N, n, dtype):
    check_product(ml, extra, 3, N, 200, n, dtype, out_extra=extra)


@pytest.mark.parametrize("n", [20, 700])
def test_rows_that_are_not_finite_stay_alone(ml, n):
    rng = np.random.default_rng(4)
    w, ws = weights(rng, 2, 130, 300)
    x = torch.randn((n, 300), device=DEV).to(torch.bfloat16)
    route = ml.make_fp8_route(dev(w), dev(ws))
    off = dev(np.array([0, n // 2, n], dtype=np.int32))
    outs = []
    for bad in (False, True):
        if bad:
            x[3, 5], x[n // 2, 299], x[n - 1, 0] = float("inf"), float("nan"), -float("inf")
        q, s = quantised(ml, x)
        out = torch.empty((n, 130), device=DEV, dtype=torch.bfloat16)
        ml.mlora_fp8_gemm(route, q, s, out, off)
        outs.append(out)
    hit = torch.zeros(n, dtype=torch.bool, device=DEV)
    hit[[3, n // 2, n - 1]] = True
    assert torch.equal(outs[0][~hit], outs[1][~hit])
    assert outs[1][hit].isnan().all()


@pytest.mark.parametrize("offsets", [[5, 2, 9, 40], [-4, 3, 3, 1000], [0, 0, 0, 0],
                                     [20, 10, 5, 0], [2 ** 31 - 1] * 4])
@pytest.mark.parametrize("n", [20, 400])
def test_strange_offsets_stay_in_bounds(ml, offsets, n):
    """Nothing outside the out rows is written, whatever the offsets hold."""
    rng = np.random.default_rng(5)
    w, ws = weights(rng, 3, 40, 200)
    route = ml.make_fp8_route(dev(w), dev(ws))
    q, s = quantised(ml, torch.randn((n, 200), device=DEV))
    held = torch.full((n + 2, 56), 3.0, device=DEV, dtype=torch.bfloat16)
    ml.mlora_fp8_gemm(route, q, s, held[1:n + 1, 8:48], dev(np.array(offsets, dtype=np.int32)))
    held[1:n + 1, 8:48] = 3.0
    assert (held == 3).all()


def test_gradient_of_rows_against_the_forward(ml):
    """<W q, g> = <q, W^T g> with the transposed route of the same weights, exactly
    quantised rows: both sides within their bounds."""
    rng = np.random.default_rng(6)
    E, N, K, n = 3, 150, 260, 80
    w, ws = weights(rng, E, N, K)
    full = fp8.expand(w, ws)
    off = spans(rng, n, E)
    rows = {k: fp8.quantise(rng.normal(0, 1, (n, k)), whole(k)) for k in (N, K)}
    got, ref = {}, {}
    for k, transpose in ((K, False), (N, True)):
        codes, s = rows[k][0], rows[k][1].astype(np.float32)
        out = torch.empty((n, N + K - k), device=DEV)
        ml.mlora_fp8_gemm(ml.make_fp8_route(dev(w), dev(ws), transpose=transpose),
                          rows_in(ml, codes), dev(s), out, dev(off))
        got[k], ref[k] = to64(out), fp8.rows_of(codes, s, k)
    lhs, rhs = (got[K] * ref[N]).sum(1), (got[N] * ref[K]).sum(1)
    mag = np.zeros(n)
    for e in range(E):
        sl = slice(off[e], off[e + 1])
        mag[sl] = ((np.abs(ref[K][sl]) @ np.abs(full[e]).T) * np.abs(ref[N][sl])).sum(1)
    close(lhs, rhs, mag * (N + K + 16) * F32)


@pytest.mark.parametrize("n", [30, 600])
def test_streams_graphs_and_reruns(ml, n):
    """A side stream, a rerun and replays of a captured graph (with eager work
    between them, and inputs changed in place) give the eager bits."""
    rng = np.random.default_rng(7)
    E, N, K = 6, 140, 300
    w, ws = weights(rng, E, N, K)
    route = ml.make_fp8_route(dev(w), dev(ws))
    x = torch.randn((n, K), device=DEV).to(torch.bfloat16)
    off = dev(spans(rng, n, E))
    q, s = quantised(ml, x)
    out = torch.zeros((n, N), device=DEV, dtype=torch.bfloat16)

    def step(stream=None):
        ml.mlora_fp8_quant(x, q, s, stream=stream)
        ml.mlora_fp8_gemm(route, q, s, out, off, stream=stream)

    step()
    want = out.clone()
    side = torch.cuda.Stream()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(torch.randn((n, K), device=DEV))
        off.copy_(dev(spans(rng, n, E)))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        assert torch.equal(out, got), i


def test_python_refuses(ml):
    x = torch.zeros((4, 300), device=DEV)
    q, s = quantised(ml, x)
    route = ml.make_fp8_route(torch.zeros((2, 100, 300), dtype=torch.uint8, device=DEV),
                              torch.ones((2, 1, 3), device=DEV))
    out, off = torch.zeros((4, 100), device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    cases = [
        (TypeError, lambda: ml.mlora_fp8_quant(x.half(), q, s)),
        (TypeError, lambda: ml.mlora_fp8_quant(x, q.int(), s)),
        (TypeError, lambda: ml.mlora_fp8_quant(x, q, s.double())),
        (TypeError, lambda: ml.mlora_fp8_quant(x, q, s, up=x.bfloat16())),
        (ValueError, lambda: ml.mlora_fp8_quant(x, q[:, :300], s)),
        (ValueError, lambda: ml.mlora_fp8_quant(x, q, s[:2])),
        (ValueError, lambda: ml.mlora_fp8_quant(x, q, s, up=x[:3])),
        (ValueError, lambda: ml.mlora_fp8_quant(x.cpu(), q, s)),
        (ValueError, lambda: ml.mlora_fp8_quant(x.t(), q, s)),
        (ValueError, lambda: ml.mlora_fp8_gemm(route, q[:, :128], s, out, off)),
        (ValueError, lambda: ml.mlora_fp8_gemm(route, q, s, out[:, :99], off)),
        (ValueError, lambda: ml.mlora_fp8_gemm(route, q, s, out, off[:2])),
        (TypeError, lambda: ml.mlora_fp8_gemm(route, q, s, out, off.long())),
        (TypeError, lambda: ml.mlora_fp8_gemm(route, q, s, out.half(), off)),
        (ValueError, lambda: ml.mlora_fp8_gemm(route, q, s, out, off, off)),
        (ml.MloraError, lambda: ml.mlora_fp8_gemm(route, q, s, out)),
        (ValueError, lambda: ml.make_fp8_route(q, s)),
        (TypeError, lambda: ml.make_fp8_route(x.view(1, 4, 300), torch.ones((1, 1, 3), device=DEV))),
        (ValueError, lambda: ml.make_fp8_route(q.view(1, 4, -1), torch.ones((1, 1, 2), device=DEV))),
    ]
    for error, call in cases:
        with pytest.raises(error):
            call()


def test_packed_memory_belongs_to_the_given_stream(ml):
    """As make_w4_route: a dropped route's block goes back to the stream that wrote it."""
    w = torch.zeros((8, 2048, 2048), dtype=torch.uint8, device=DEV)
    s = torch.ones((8, 16, 16), device=DEV)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    route = ml.make_fp8_route(w, s, stream=side)
    at, size = route._keep.data_ptr(), route._keep.numel()
    torch.cuda.synchronize()
    del route
    here = torch.empty(size, dtype=torch.uint8, device=DEV)
    assert here.data_ptr() != at
    torch.cuda.synchronize()
