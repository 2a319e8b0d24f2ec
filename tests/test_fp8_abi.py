"""Host side of the 8-bit products, the layer of a few tokens and the norms around
a block (no GPU): what each entry point refuses before anything is enqueued, the
size queries, calls with nothing to do, and the fp64 forms against the formats'
definitions and against central differences."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import moe_expert_lora_amd as ml
from oracle import fp8

P = 0x10000  # a non-null, 256-byte aligned address; a refused call never reads it
BF16, F32 = ml.MLORA_BF16, ml.MLORA_F32
INVALID, CAPACITY, OK = ml.MLORA_ERR_INVALID, ml.MLORA_ERR_CAPACITY, ml.MLORA_OK


@pytest.fixture(scope="module")
def lib():
    return ml.load()


def _call(lib, name, base, **changed):
    args = dict(base)
    assert set(changed) <= set(args), changed
    args.update(changed)
    return getattr(lib, name)(*args.values())


def _refused(lib, name, base, bad, code=INVALID):
    assert _call(lib, name, base, **bad) == code
    assert lib.mlora_last_error().decode().startswith(name + ":")


PACK = dict(w=P, scales=P, E=4, k=256, n=100, transpose=0, packed=P, nbytes=1 << 40, route=None,
            stream=None)
PACK_BAD = [dict(E=0), dict(E=1025), dict(k=0), dict(k=(1 << 20) + 1), dict(n=0), dict(n=1 << 21),
            dict(w=None), dict(scales=None), dict(packed=None), dict(packed=P + 16)]


@pytest.mark.parametrize("bad", PACK_BAD, ids=str)
def test_pack_refuses(lib, bad):
    r = ml.Fp8Route()
    _refused(lib, "mlora_fp8_pack", {**PACK, "route": ctypes.byref(r)}, bad)


def test_pack_sizes(lib):
    # 8 column tiles of 16 (one block of 128), 2 blocks of k; a scale a block
    assert ml.mlora_fp8_packed_bytes(4, 256, 100) == 4 * 8 * 2 * 2048 + 256
    assert ml.mlora_fp8_packed_bytes(1, 1, 1) == 8 * 2048 + 256
    assert ml.mlora_fp8_packed_bytes(0, 256, 100) == 0
    assert ml.mlora_fp8_packed_bytes(4, 256, (1 << 20) + 1) == 0
    assert [ml.mlora_fp8_row_width(k) for k in (0, 1, 128, 129, 1 << 20, (1 << 20) + 1)] == \
        [0, 128, 128, 384, (1 << 20) + 128, 0]
    r = ml.Fp8Route()
    base = {**PACK, "route": ctypes.byref(r)}
    _refused(lib, "mlora_fp8_pack", base,
             dict(nbytes=ml.mlora_fp8_packed_bytes(4, 256, 100) - 1), CAPACITY)
    _refused(lib, "mlora_fp8_pack", {**base, "route": None}, {})


QUANT = dict(x=P, x_ld=300, up=None, up_ld=0, dtype=BF16, n=4, k=300, q=P, q_ld=384, scales=P,
             stream=None)
QUANT_BAD = [dict(dtype=2), dict(n=-1), dict(n=1 << 30), dict(k=0), dict(k=(1 << 20) + 1),
             dict(x_ld=299), dict(up=P, up_ld=299), dict(q_ld=368), dict(q_ld=392), dict(x=None),
             dict(q=None), dict(scales=None), dict(q=P + 8)]


@pytest.mark.parametrize("bad", QUANT_BAD, ids=str)
def test_quant_refuses(lib, bad):
    _refused(lib, "mlora_fp8_quant", QUANT, bad)


GEMM = dict(route=None, q=P, q_rows=4, q_ld=384, scales=P, out=P, out_ld=100, dtype=BF16, n=8,
            offsets=P, ids=P, k=2, stream=None)
GEMM_BAD = [dict(dtype=2), dict(n=-1), dict(n=1 << 30), dict(q_rows=-1), dict(q_rows=1 << 30),
            dict(k=0), dict(k=1025), dict(offsets=None), dict(ids=None), dict(q_ld=256),
            dict(q_ld=385), dict(out_ld=99), dict(q=None), dict(scales=None), dict(out=None),
            dict(q=P + 4), dict(route=None)]


@pytest.mark.parametrize("bad", GEMM_BAD, ids=str)
def test_gemm_refuses(lib, bad):
    r = ml.Fp8Route(P, P, 4, 300, 100)
    _refused(lib, "mlora_fp8_gemm", {**GEMM, "route": ctypes.byref(r)}, bad)


@pytest.mark.parametrize("route", [(None, P, 4, 300, 100), (P, None, 4, 300, 100),
                                   (P + 4, P, 4, 300, 100), (P, P, 0, 300, 100),
                                   (P, P, 4, 0, 100), (P, P, 4, 300, 1 << 21)], ids=str)
def test_gemm_refuses_routes(lib, route):
    r = ml.Fp8Route(*route)
    _refused(lib, "mlora_fp8_gemm", {**GEMM, "route": ctypes.byref(r)}, {})


LAYER = dict(gate=None, up=None, down=None, x=P, x_ld=256, dtype=BF16, n=4, logits=P,
             logits_ld=8, k=2, renorm=1, out=P, out_ld=256, indices=P, weights=P, ws=P,
             nbytes=1 << 40, stream=None)
LAYER_BAD = [dict(dtype=2), dict(n=-1), dict(n=17), dict(k=0), dict(k=9), dict(x_ld=255),
             dict(out_ld=255), dict(logits_ld=7), dict(x=None), dict(logits=None), dict(out=None),
             dict(ws=P + 8), dict(gate=None), dict(up=None), dict(down=None)]


def _layer_routes(gate=(8, 256, 100), up=(8, 256, 100), down=(8, 100, 256)):
    rs = [ml.Fp8Route(P, P, *s) for s in (gate, up, down)]
    return dict(zip(("gate", "up", "down"), map(ctypes.pointer, rs)))


@pytest.mark.parametrize("bad", LAYER_BAD, ids=str)
def test_layer_refuses(lib, bad):
    _refused(lib, "mlora_moe_layer", {**LAYER, **_layer_routes()}, bad)


@pytest.mark.parametrize("bad", [dict(up=(8, 256, 99)), dict(up=(8, 255, 100)),
                                 dict(down=(8, 100, 255)), dict(down=(8, 99, 256)),
                                 dict(down=(7, 100, 256)), dict(gate=(0, 256, 100))], ids=str)
def test_layer_refuses_routes(lib, bad):
    _refused(lib, "mlora_moe_layer", {**LAYER, **_layer_routes(**bad)}, {})


def test_layer_workspace(lib):
    need = ml.mlora_moe_layer_workspace_bytes(4, 8, 2, 256, 100)
    assert need > 0
    base = {**LAYER, **_layer_routes()}
    _refused(lib, "mlora_moe_layer", base, dict(nbytes=need - 1), CAPACITY)
    _refused(lib, "mlora_moe_layer", base, dict(ws=None), CAPACITY)
    for bad in ((0, 8, 2, 256, 100), (17, 8, 2, 256, 100), (4, 0, 2, 256, 100),
                (4, 8, 9, 256, 100), (4, 8, 2, 0, 100)):
        assert ml.mlora_moe_layer_workspace_bytes(*bad) == 0


def _block(**changed):
    f = dict(residual=P, residual_ld=64, y=P, y_ld=64, x_weight=P, y_weight=P, gate=P, gate_ld=64,
             gate_form=3, dtype=BF16, w_dtype=F32, dim=64, n_tokens=4, residual_scale=1.0,
             y_scale=1.0, weight_offset=0.0, eps=1e-6)
    assert set(changed) <= set(f)
    return ml.NormBlock(*{**f, **changed}.values())


BLOCK_BAD = [dict(dtype=2), dict(w_dtype=2), dict(n_tokens=-1), dict(n_tokens=1 << 30),
             dict(dim=0), dict(dim=16385, residual_ld=20000, y_ld=20000, gate_ld=20000),
             dict(gate_form=4), dict(gate_form=-1), dict(eps=-1e-6), dict(eps=float("nan")),
             dict(eps=float("inf")), dict(residual_ld=63), dict(y_ld=63), dict(gate_ld=63),
             dict(gate_form=2, gate_ld=0), dict(residual=None), dict(gate=None),
             dict(gate_form=1, gate=None), dict(y=None), dict(y=None, gate_form=0)]
FORWARD = dict(block=None, r=P, r_ld=64, x=2 * P, x_ld=64, stream=None)
BACKWARD = dict(block=None, d_r=P, d_r_ld=64, d_x=P, d_x_ld=64, d_res=P, d_res_ld=64, d_y=P,
                d_y_ld=64, d_wx=P, d_wy=P, d_gate=P, d_gate_ld=64, ws=P, nbytes=1 << 40,
                stream=None)


@pytest.mark.parametrize("bad", BLOCK_BAD, ids=str)
def test_norm_refuses_blocks(lib, bad):
    b = _block(**bad)
    _refused(lib, "mlora_block_norm", {**FORWARD, "block": ctypes.byref(b)}, {})
    _refused(lib, "mlora_block_norm_backward", {**BACKWARD, "block": ctypes.byref(b)}, {})


@pytest.mark.parametrize("bad", [dict(r=None, x=None), dict(r_ld=63), dict(x_ld=63), dict(x=P),
                                 dict(block=None)], ids=str)
def test_norm_forward_refuses(lib, bad):
    b = _block()
    _refused(lib, "mlora_block_norm", {**FORWARD, "block": ctypes.byref(b)}, bad)


@pytest.mark.parametrize("changed,bad", [
    ({}, dict(d_r=None, d_x=None)), ({}, dict(d_r_ld=63)), ({}, dict(d_x_ld=63)),
    ({}, dict(d_res_ld=63)), ({}, dict(d_y_ld=63)), ({}, dict(d_gate_ld=63)),
    (dict(gate_form=2, gate_ld=1), dict(d_gate_ld=0)), (dict(gate_form=0), {}),
    (dict(y_weight=None), {}), ({}, dict(ws=P + 8)), ({}, dict(block=None)),
    (dict(y=None, y_weight=None, gate_form=0), dict(d_gate=None, d_wy=None))], ids=str)
def test_norm_backward_refuses(lib, changed, bad):
    b = _block(**changed)
    _refused(lib, "mlora_block_norm_backward", {**BACKWARD, "block": ctypes.byref(b)}, bad)


def test_norm_workspace(lib):
    need = ml.mlora_block_norm_backward_workspace_bytes(4, 64)
    assert need % 256 == 0 and need >= 3 * 64 * 4  # three sums, of one workgroup at least
    b = _block()
    base = {**BACKWARD, "block": ctypes.byref(b)}
    _refused(lib, "mlora_block_norm_backward", base, dict(nbytes=need - 1), CAPACITY)
    _refused(lib, "mlora_block_norm_backward", base, dict(ws=None), CAPACITY)
    for bad in ((0, 64), (-1, 64), (4, 0), (4, 16385), (1 << 30, 64)):
        assert ml.mlora_block_norm_backward_workspace_bytes(*bad) == 0
    # bounded, whatever the number of tokens
    assert ml.mlora_block_norm_backward_workspace_bytes(1 << 29, 16384) <= 3 * 1024 * 16384 * 4


def test_nothing_to_do(lib):
    r = ml.Fp8Route(P, P, 4, 300, 100)
    null = lambda base: {k: None if v == P else v for k, v in base.items()}  # noqa: E731
    assert _call(lib, "mlora_fp8_quant", null(QUANT), n=0) == OK
    assert _call(lib, "mlora_fp8_gemm", {**null(GEMM), "offsets": P, "ids": P}, n=0,
                 route=ctypes.byref(r)) == OK
    # no rows to read from: every row is left as it was
    assert _call(lib, "mlora_fp8_gemm", {**null(GEMM), "offsets": P, "ids": P}, q_rows=0,
                 route=ctypes.byref(r)) == OK
    assert _call(lib, "mlora_moe_layer", {**null(LAYER), **_layer_routes()}, n=0) == OK
    b = _block(n_tokens=0, residual=None, gate=None)
    assert _call(lib, "mlora_block_norm", {**null(FORWARD), "x": None},
                 block=ctypes.byref(b)) == OK
    assert _call(lib, "mlora_block_norm_backward", null(BACKWARD), block=ctypes.byref(b)) == OK
    assert lib.mlora_last_error() == b""


def test_sizes_past_32_bits_are_refused():
    for call in (lambda: ml.mlora_fp8_packed_bytes(1, 1 << 32, 1),
                 lambda: ml.mlora_fp8_row_width((1 << 32) + 8),
                 lambda: ml.mlora_moe_layer_workspace_bytes(1, (1 << 32) + 8, 1, 1, 1),
                 lambda: ml.mlora_block_norm_backward_workspace_bytes(1, (1 << 32) + 8)):
        with pytest.raises(ValueError):
            call()


# -- the fp64 forms ----------------------------------------------------------

def test_e4m3_against_torch():
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8.e4m3_decode(codes), want, equal_nan=True)
    v = np.concatenate([np.random.default_rng(0).normal(0, s, 4000).astype(np.float32)
                        for s in (0.001, 0.05, 1, 100)])
    table = fp8.e4m3_values()
    v = np.concatenate([v, (table[1:] + table[:-1]) / 2, -(table[1:] + table[:-1]) / 2, table])
    v = v[np.abs(v) <= 448].astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = fp8.e4m3_round(v)
    assert np.array_equal(got[v != 0], want[v != 0])


def test_quantise_by_hand():
    # m = 448: scale 1; 17 lies half way between 16 and 18, 19 between 18 and 20
    x = np.zeros((1, 130))
    x[0, :5] = [448, 17, 19, -17, 2.0 ** -10]
    x[0, 129] = 7.0  # the next group: scale 1 / 64, code 448
    codes, scales = fp8.quantise(x, 256)
    assert scales.shape == (2, 1) and scales[0, 0] == 1 and scales[1, 0] == 7 / 448
    assert fp8.e4m3_decode(codes[0, :5]).tolist() == [448, 16, 20, -16, 0]
    assert fp8.e4m3_decode(codes[0, 129]) == 448 and not codes[0, 130:].any()
    codes, scales = fp8.quantise(np.array([[1.0, np.inf]]), 128)
    assert np.isnan(scales).all() and not codes.any()


NORMS = [dict(), dict(y=True), dict(y=True, y_weight=True), dict(y=True, gate=(5,)),
         dict(y=True, y_weight=True, gate=(4, 1), x_weight=True),
         dict(y=True, y_weight=True, gate=(4, 5), x_weight=True, offset=1.0)]


@pytest.mark.parametrize("case", NORMS, ids=str)
def test_norm_gradient_against_differences(case):
    rng = np.random.default_rng(1)
    ins = {"residual": rng.normal(size=(4, 5))}
    shapes = dict(y=(4, 5), y_weight=(5,), x_weight=(5,), gate=case.get("gate"))
    for name in ("y", "x_weight", "y_weight", "gate"):
        if case.get(name):
            ins[name] = rng.normal(size=shapes[name])
    kw = dict(residual_scale=0.7, y_scale=1.3, offset=case.get("offset", 0.0), eps=1e-3)
    d_r, d_x = rng.normal(size=(2, 4, 5))

    def loss(v):
        r, x = fp8.block_norm(**v, **kw)
        return (d_r * r).sum() + (d_x * x).sum()

    got = fp8.block_norm_gradient(d_r=d_r, d_x=d_x, **ins, **kw)
    step = 1e-5
    for name, v in ins.items():
        for at in np.ndindex(v.shape):
            up, dn = v.copy(), v.copy()
            up[at] += step
            dn[at] -= step
            diff = (loss({**ins, name: up}) - loss({**ins, name: dn})) / (2 * step)
            assert abs(diff - got[name][at]) < 1e-7, (name, at)


def test_layer_form_is_the_calls_one_by_one():
    from oracle import moe
    rng = np.random.default_rng(2)
    E, dim, hidden, T, k = 5, 6, 4, 3, 2
    gate, up = rng.normal(size=(2, E, hidden, dim))
    down = rng.normal(size=(E, dim, hidden))
    x, logits = rng.normal(size=(T, dim)), rng.normal(size=(T, E))
    out, idx, w, _ = fp8.layer(x, logits, gate, up, down, k, True)
    ids = idx.reshape(-1)
    g, u = (moe.w4_products(m, x, ids, k, False, T * k) for m in (gate, up))
    rows = moe.w4_products(down, fp8.silu(g) * u, ids, k, True, T * k)
    assert np.allclose(out, moe.combine(rows, T, k, w, None)[0], rtol=0, atol=1e-12)
