"""Host side of the MoE layer's operators (no GPU): what each entry point
refuses before anything is enqueued, the size queries, calls with nothing to
do, and the fp64 forms against central differences."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import moe_expert_lora_amd as ml
from oracle import moe

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


ROUTER = dict(logits=P, ld=128, dtype=BF16, n=4, E=128, k=8, renorm=1, indices=P, weights=P,
              stream=None)
ROUTER_BWD = dict(logits=P, ld=128, dtype=BF16, n=4, E=128, k=8, renorm=1, indices=P, dw=P, dl=P,
                  dl_ld=128, stream=None)
SORT = dict(ids=P, n=8, E=4, offsets=P, sorted_ids=P, slot_rows=P, ws=None, ws_bytes=0,
            stream=None)
DISPATCH = dict(x=P, x_ld=64, dtype=BF16, n=4, dim=64, k=2, sorted_ids=P, slot_rows=P, rows=P,
                rows_ld=64, stream=None)
COMBINE = dict(rows=P, rows_ld=64, n_rows=8, dtype=BF16, n=4, dim=64, k=2, weights=P, slot_rows=P,
               out=P, out_ld=64, stream=None)
COMBINE_BWD = dict(d_out=P, d_out_ld=64, rows=P, rows_ld=64, dtype=BF16, n=4, dim=64, k=2,
                   weights=P, slot_rows=P, sorted_ids=P, d_rows=P, d_rows_ld=64, d_weights=P,
                   stream=None)

REFUSED = [
    ("mlora_router_topk", ROUTER, [
        dict(dtype=2), dict(n=-1), dict(n=1 << 30), dict(E=0), dict(E=1025, ld=2000), dict(k=0),
        dict(k=65), dict(E=4, k=5), dict(ld=127), dict(logits=None), dict(indices=None),
        dict(weights=None)]),
    ("mlora_router_topk_backward", ROUTER_BWD, [
        dict(dtype=-1), dict(n=-1), dict(E=0), dict(k=0), dict(ld=64), dict(dl_ld=127),
        dict(logits=None), dict(indices=None), dict(dw=None), dict(dl=None)]),
    ("mlora_moe_sort", SORT, [
        dict(n=-1), dict(n=1 << 30), dict(E=0), dict(E=1025), dict(ids=None),
        dict(offsets=None), dict(sorted_ids=None), dict(slot_rows=None), dict(ws_bytes=4),
        dict(ws=P + 2, ws_bytes=64), dict(n=0, offsets=None)]),
    ("mlora_moe_dispatch", DISPATCH, [
        dict(dtype=2), dict(n=-1), dict(k=0), dict(k=65), dict(n=1 << 29, k=4), dict(dim=0),
        dict(x_ld=63), dict(rows_ld=63), dict(x=None), dict(sorted_ids=None),
        dict(slot_rows=None), dict(rows=None)]),
    ("mlora_moe_combine", COMBINE, [
        dict(dtype=2), dict(n=-1), dict(k=0), dict(dim=0), dict(rows_ld=63), dict(out_ld=63),
        dict(n_rows=-1), dict(slot_rows=None, n_rows=7), dict(rows=None), dict(out=None)]),
    ("mlora_moe_combine_backward", COMBINE_BWD, [
        dict(dtype=2), dict(n=-1), dict(k=0), dict(dim=0), dict(rows_ld=63), dict(d_out_ld=63),
        dict(d_rows_ld=63), dict(slot_rows=None), dict(sorted_ids=None), dict(d_out=None),
        dict(rows=None), dict(d_rows=None)]),
]


@pytest.mark.parametrize("name,base,bad", [(n, b, c) for n, b, cs in REFUSED for c in cs],
                         ids=[f"{n}-{c}" for n, b, cs in REFUSED for c in cs])
def test_refuses(lib, name, base, bad):
    assert _call(lib, name, base, **bad) == INVALID
    assert lib.mlora_last_error().decode().startswith(name + ":")


@pytest.mark.parametrize("name,base", [(n, b) for n, b, _ in REFUSED if n != "mlora_moe_sort"])
def test_no_tokens_is_no_work(lib, name, base):
    null = {k: None for k, v in base.items() if v == P}
    assert _call(lib, name, base, n=0, **null) == OK
    assert lib.mlora_last_error() == b""


def test_sort_workspace(lib):
    assert ml.mlora_moe_sort_workspace_bytes(0, 128) == 0
    assert ml.mlora_moe_sort_workspace_bytes(-1, 128) == 0
    assert ml.mlora_moe_sort_workspace_bytes(640, 128) == 0
    assert ml.mlora_moe_sort_workspace_bytes(1 << 30, 128) == 0  # refused
    need = ml.mlora_moe_sort_workspace_bytes(100000, 128)
    assert need > 0 and need % 256 == 0
    assert _call(lib, "mlora_moe_sort", SORT, n=100000, E=128, ws=P, ws_bytes=need - 1) == CAPACITY
    assert _call(lib, "mlora_moe_sort", SORT, n=100000, E=128) == CAPACITY
    # the size stays bounded: a count per block and expert
    assert ml.mlora_moe_sort_workspace_bytes((1 << 30) - 1, 1024) <= 256 * 1025 * 4 + 256


W4 = dict(E=4, k_in=256, n_out=100, group=64, dtype=BF16)
W4_BAD = [dict(E=0), dict(E=1025), dict(k_in=0), dict(k_in=12), dict(n_out=0), dict(group=0),
          dict(group=16), dict(group=96), dict(group=200), dict(dtype=2), dict(dtype=-1)]


@pytest.mark.parametrize("bad", W4_BAD, ids=[str(b) for b in W4_BAD])
def test_w4_refuses_weights(lib, bad):
    d = {**W4, **bad}
    assert lib.mlora_w4_packed_bytes(d["E"], d["k_in"], d["n_out"], d["group"], d["dtype"], 1) == 0
    r = ml.W4Route()
    assert lib.mlora_w4_pack(P, P, P, d["E"], d["k_in"], d["n_out"], d["group"], d["dtype"], P,
                             1 << 40, ctypes.byref(r), None) == INVALID
    r = ml.W4Route(P, P, None, d["E"], d["k_in"], d["n_out"], d["group"], d["dtype"])
    assert lib.mlora_w4_gather_gemv(ctypes.byref(r), P, 4, 1 << 21, 0, P, 1 << 21, P, 4, 1,
                                    None) == INVALID


def test_w4_packed_bytes(lib):
    # 4 pairs of column tiles of 16, 8 k steps of 512 bytes; 4 groups of 32 columns
    w, s, z = 4 * 4 * 8 * 512, 4 * 4 * 4 * 32 * 2, 4 * 4 * 4 * 32
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    assert ml.mlora_w4_packed_bytes(4, 256, 100, 64, BF16, False) == up(w) + up(s)
    assert ml.mlora_w4_packed_bytes(4, 256, 100, 64, BF16, True) == up(w) + up(s) + up(z)
    need = ml.mlora_w4_packed_bytes(4, 256, 100, 64, BF16, True)
    r = ml.W4Route()
    args = [4, 256, 100, 64, BF16]
    assert lib.mlora_w4_pack(P, P, P, *args, P, need - 1, ctypes.byref(r), None) == CAPACITY
    assert lib.mlora_w4_pack(P, P, P, *args, P + 16, need, ctypes.byref(r), None) == INVALID
    assert lib.mlora_w4_pack(None, P, P, *args, P, need, ctypes.byref(r), None) == INVALID
    assert lib.mlora_w4_pack(P, None, P, *args, P, need, ctypes.byref(r), None) == INVALID
    assert lib.mlora_w4_pack(P, P, P, *args, None, need, ctypes.byref(r), None) == INVALID
    assert lib.mlora_w4_pack(P, P, P, *args, P, need, None, None) == INVALID


GEMV = dict(x=P, x_rows=4, x_ld=256, by_row=0, out=P, out_ld=100, ids=P, n_rows=8, k=2,
            stream=None)
GEMV_BAD = [dict(k=0), dict(n_rows=-1), dict(n_rows=1 << 30), dict(x_rows=3),
            dict(by_row=1, x_rows=7), dict(x_ld=248), dict(x_ld=257), dict(out_ld=99),
            dict(ids=None), dict(x=None), dict(out=None), dict(x=P + 8),
            dict(x_rows=1 << 24, n_rows=1 << 25), dict(x_ld=1 << 40)]


@pytest.mark.parametrize("bad", GEMV_BAD, ids=[str(b) for b in GEMV_BAD])
def test_w4_gemv_refuses(lib, bad):
    r = ml.W4Route(P, P, None, 4, 256, 100, 64, BF16)
    args = {**GEMV, **bad}
    assert lib.mlora_w4_gather_gemv(ctypes.byref(r), *args.values()) == INVALID
    assert lib.mlora_last_error().decode().startswith("mlora_w4_gather_gemv:")


def test_w4_gemv_no_rows_and_null_route(lib):
    r = ml.W4Route(P, P, None, 4, 256, 100, 64, BF16)
    args = {**GEMV, **dict(n_rows=0, x_rows=0, x=None, out=None, ids=P)}
    assert lib.mlora_w4_gather_gemv(ctypes.byref(r), *args.values()) == OK
    assert lib.mlora_w4_gather_gemv(None, *GEMV.values()) == INVALID
    r = ml.W4Route(None, P, None, 4, 256, 100, 64, BF16)
    assert lib.mlora_w4_gather_gemv(ctypes.byref(r), *GEMV.values()) == INVALID


# ---------------------------------------------------------------------------
# the Python functions
# ---------------------------------------------------------------------------

def test_python_functions_take_device_tensors():
    """Host tensors and other objects are refused before anything is called."""
    torch = pytest.importorskip("torch")
    x, i = torch.zeros((4, 8)), torch.zeros(4, dtype=torch.int32)
    route = ml.W4Route(P, P, None, 1, 8, 8, 32, F32)
    calls = [lambda t: ml.mlora_router_topk(t, i, x),
             lambda t: ml.mlora_router_topk_backward(t, i, x, x),
             lambda t: ml.mlora_moe_sort(t, 3, i, i, i),
             lambda t: ml.mlora_moe_dispatch(t, x, i, i, 1),
             lambda t: ml.mlora_moe_combine(t, x, 1),
             lambda t: ml.mlora_moe_combine_backward(t, x, x, x, x, 1),
             lambda t: ml.mlora_w4_gather_gemv(route, t, x)]
    for call in calls:
        with pytest.raises(ValueError, match="must be a device tensor"):
            call(x)
        with pytest.raises(TypeError, match="must be a tensor"):
            call([1.0])
    assert route.address == ctypes.addressof(route)


# ---------------------------------------------------------------------------
# the fp64 forms themselves
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_against_differences(renorm):
    rng = np.random.default_rng(3)
    lg = rng.normal(size=(3, 9))
    idx = moe.router_choice(lg, 4)
    dw = rng.normal(size=(3, 4))
    grad = moe.router_gradient(lg, idx, dw, renorm)
    h = 1e-5
    for t in range(3):
        for e in range(9):
            up, down = lg.copy(), lg.copy()
            up[t, e] += h
            down[t, e] -= h
            num = ((moe.router_weights(up, idx, renorm) - moe.router_weights(down, idx, renorm))
                   * dw).sum() / (2 * h)
            assert abs(num - grad[t, e]) <= 1e-9


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(4)
    n, k, dim = 4, 3, 5
    ids = np.array([0, 2, 1, -1, 1, 0, 2, 2, 0, 1, 0, 7], dtype=np.int32)
    _, _, slots = moe.sort_by_expert(ids, 3)
    rows, w = rng.normal(size=(n * k, dim)), rng.normal(size=(n, k))
    g = rng.normal(size=(n, dim))
    d_rows, d_w, _ = moe.combine_gradient(g, rows, k, w, slots)
    f = lambda r, v: (moe.combine(r, n, k, v, slots)[0] * g).sum()  # noqa: E731
    h = 1e-4
    for a, d in ((rows, d_rows), (w, d_w)):
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + h
            up = f(rows, w)
            a[i] = old - h
            down = f(rows, w)
            a[i] = old
            assert abs((up - down) / (2 * h) - d[i]) <= 1e-9


def test_sort_definition():
    off, order, rows = moe.sort_by_expert(np.array([2, 0, -1, 2, 5, 0]), 3)
    assert off.tolist() == [0, 2, 2, 4]
    assert order.tolist() == [1, 5, 0, 3, -1, -1]
    assert rows.tolist() == [2, 0, -1, 3, -1, 1]
