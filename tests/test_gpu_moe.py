"""GPU tests of the MoE layer's row operators (router choice and gradient,
sort by expert, dispatch, combine and its gradient) against their fp64 forms.

Tolerances, derived from the formulas (u = 2^-24 per fp32 rounding, 2^-8 of
the value for one bf16 rounding):
* router weight p = exp(l - max) / sum: the rounded difference d = l - max
  moves the exponential by |d| u, expf, the sum over a lane's values and the
  lanes (at most 16 + 10 additions) and the division the rest: relative
  (|d| + 64) u, plus the smallest normal number.
* router gradient p (dw - dot): each factor as above, the difference
  absolutely: p (|dw| + sum |dw| p) (|d| + 64) 2 u.
* combine: k products and additions of fp32: (k + 1) u sum |w x|.
* d_weights: a lane adds dim / 64 + 8 products, then 9 partial sums are added:
  (dim / 64 + 24) u sum |d x|; d_rows: one product, u.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import moe

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 2.0 ** -126


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(scope="module")
def ml():
    import moe_expert_lora_amd
    return moe_expert_lora_amd


def _np(t):
    return t.detach().double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _close(got, ref, tol, half, what):
    lim = tol + half * (np.abs(ref) + tol) + TINY
    bad = np.abs(got - ref) > lim
    assert np.isfinite(got).all(), what
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------

def _route(ml, lg, k, renorm, **kw):
    idx = torch.full((lg.shape[0], k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((lg.shape[0], k), 9e9, dtype=torch.float32, device=DEV)
    ml.mlora_router_topk(lg, idx, w, renormalize=renorm, **kw)
    torch.cuda.synchronize()
    return idx, w


def _check_router(ml, lg, k, renorm, backward=True):
    ref = _np(lg)
    idx, w = _route(ml, lg, k, renorm)
    want = moe.router_choice(ref, k)
    assert np.array_equal(_np(idx), want)
    wref = moe.router_weights(ref, want, renorm)
    top = ref.max(1, keepdims=True)
    d = np.where(np.isfinite(ref), np.abs(ref - np.where(np.isfinite(top), top, 0)), 0)
    span = np.take_along_axis(d, want, 1)
    _close(_np(w), wref, wref * (span + 64) * U, 0.0, "weights")
    if not backward:
        return
    g = torch.Generator(device=DEV).manual_seed(5)
    dw = torch.randn(w.shape, generator=g, device=DEV)
    dl = torch.full_like(lg, 9e9)
    ml.mlora_router_topk_backward(lg, idx, dw, dl, renormalize=renorm)
    torch.cuda.synchronize()
    gref = moe.router_gradient(ref, want, _np(dw), renorm)
    dense = np.zeros_like(ref)
    np.put_along_axis(dense, want, np.abs(_np(dw)), 1)
    p = np.zeros_like(ref)
    if renorm:
        np.put_along_axis(p, want, wref, 1)
    else:
        live = np.isfinite(top[:, 0])
        ex = np.exp(ref[live] - top[live])
        p[live] = ex / ex.sum(1, keepdims=True)
    tol = p * (dense + (dense * p).sum(1, keepdims=True)) * (d + 64) * 2 * U
    _close(_np(dl), gref, tol, HALF[lg.dtype], "d_logits")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k", [
    (1, 1, 1), (1, 2, 2), (3, 7, 3), (5, 8, 8), (80, 128, 8), (67, 100, 6), (9, 64, 1),
    (33, 128, 16), (33, 128, 17), (10, 129, 8), (10, 250, 4), (17, 256, 8), (9, 200, 32),
    (9, 200, 33), (11, 256, 64), (6, 257, 2),
    (12, 384, 6), (5, 511, 8), (5, 512, 64), (4, 513, 8), (3, 1000, 8), (3, 1024, 64), (1030, 60, 4),
    (4100, 128, 8), (6144, 256, 8), (6147, 200, 5)])
def test_router(ml, dtype, renorm, tokens, experts, top_k):
    g = torch.Generator(device=DEV).manual_seed(tokens * 7 + experts)
    lg = (torch.randn((tokens, experts), generator=g, device=DEV) * 2).to(DT[dtype])
    _check_router(ml, lg, top_k, renorm)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_router_ties_zeros_and_wide_values(ml, dtype):
    rng = np.random.default_rng(11)
    lg = rng.integers(-2, 3, size=(40, 96)).astype(np.float32)     # many equal values
    lg[3] = 0.0
    lg[4] = np.where(np.arange(96) % 2, 0.0, -0.0)                 # -0 equals +0
    lg[5] = rng.normal(size=96) * 50                               # probabilities down to 0
    lg[6] = -1e30
    lg[7, :] = 3e38
    t = torch.from_numpy(lg).to(DEV).to(DT[dtype])
    _check_router(ml, t, 8, False)
    _check_router(ml, t, 8, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("experts", [24, 200])
def test_router_masked_experts(ml, dtype, experts):
    """-inf masks: chosen last with weight 0; a row with nothing else gets the
    first experts, weights of 0 and a gradient of 0."""
    rng = np.random.default_rng(12)
    lg = rng.normal(size=(6, experts)).astype(np.float32)
    lg[0] = -np.inf
    lg[1, : experts - 3] = -np.inf
    lg[2, 3:] = -np.inf
    lg[3, ::2] = -np.inf
    lg[4] = np.finfo(np.float32).min if dtype == "f32" else -3.3895314e38  # the lowest value
    t = torch.from_numpy(lg).to(DEV).to(DT[dtype])
    for renorm in (False, True):
        idx, w = _route(ml, t, 6, renorm)
        assert _np(idx)[0].tolist() == list(range(6))
        assert (_np(w)[0] == 0).all() and (_np(w)[1, 3:] == 0).all()
        with np.errstate(invalid="ignore"):
            _check_router(ml, t, 6, renorm)


def test_router_nan_and_infinity_stay_in_their_row(ml):
    g = torch.Generator(device=DEV).manual_seed(13)
    for dtype in (torch.bfloat16, torch.float32):
        lg = torch.randn((8, 128), generator=g, device=DEV).to(dtype)
        clean_i, clean_w = _route(ml, lg, 4, False)
        lg[2, 100] = float("nan")
        lg[2, 50] = -float("nan")
        lg[5, 9] = float("inf")
        idx, w = _route(ml, lg, 4, False)
        assert _np(idx)[2, :2].tolist() == [50, 100] and int(idx[5, 0]) == 9
        assert ((idx >= 0) & (idx < 128)).all()
        keep = [0, 1, 3, 4, 6, 7]
        assert torch.equal(idx[keep], clean_i[keep]) and torch.equal(w[keep], clean_w[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_router_strides_and_alignment(ml, dtype):
    g = torch.Generator(device=DEV).manual_seed(14)
    wide = torch.randn((30, 300), generator=g, device=DEV).to(DT[dtype])
    for lg in (wide[:, 8:136], wide[:, 3:131], wide[::2, 16:144], wide[:, 1:258]):
        _check_router(ml, lg, 8, False, backward=False)
        idx, w = _route(ml, lg, 8, True)
        dw = torch.randn(w.shape, generator=g, device=DEV)
        a = torch.zeros((lg.shape[0], 400), dtype=lg.dtype, device=DEV)
        view = a[:, 5:5 + lg.shape[1]]
        ml.mlora_router_topk_backward(lg, idx, dw, view, renormalize=True)
        b = torch.empty(lg.shape, dtype=lg.dtype, device=DEV)
        ml.mlora_router_topk_backward(lg.contiguous(), idx, dw, b, renormalize=True)
        assert torch.equal(view, b)
        assert int((a[:, :5] != 0).sum()) == 0 and int((a[:, 5 + lg.shape[1]:] != 0).sum()) == 0


def test_router_gradient_ignores_indices_out_of_range(ml):
    lg = torch.randn((2, 16), device=DEV)
    idx = torch.tensor([[3, -1], [99, 5]], dtype=torch.int32, device=DEV)
    dw = torch.ones((2, 2), device=DEV)
    dl = torch.empty_like(lg)
    ml.mlora_router_topk_backward(lg, idx, dw, dl)
    ref = np.zeros((2, 16))
    for t, e in ((0, 3), (1, 5)):
        p = np.exp(_np(lg)[t] - _np(lg)[t].max())
        p /= p.sum()
        one = np.eye(16)[e]
        ref[t] = p * (one - p[e])
    assert np.abs(_np(dl) - ref).max() <= 200 * U


def test_no_tokens(ml):
    for dt in (torch.bfloat16, torch.float32):
        lg = torch.empty((0, 16), dtype=dt, device=DEV)
        idx = torch.empty((0, 4), dtype=torch.int32, device=DEV)
        w = torch.empty((0, 4), device=DEV)
        ml.mlora_router_topk(lg, idx, w)
        ml.mlora_router_topk_backward(lg, idx, w, torch.empty_like(lg))
        off = torch.full((17,), 5, dtype=torch.int32, device=DEV)
        none = torch.empty((0,), dtype=torch.int32, device=DEV)
        ml.mlora_moe_sort(none, 16, off, none, none)
        assert int(off.abs().sum()) == 0
        x = torch.empty((0, 24), dtype=dt, device=DEV)
        ml.mlora_moe_dispatch(x, torch.empty_like(x), none, none, 4)
        ml.mlora_moe_combine(x, torch.empty_like(x), 4, w, none)
        ml.mlora_moe_combine_backward(x, x, w, torch.empty_like(x), w, 4, none, none)


# ---------------------------------------------------------------------------
# sort
# ---------------------------------------------------------------------------

def _sort(ml, ids, E):
    n = ids.numel()
    off = torch.full((E + 1,), -9, dtype=torch.int32, device=DEV)
    order = torch.full((n,), -9, dtype=torch.int32, device=DEV)
    rows = torch.full((n,), -9, dtype=torch.int32, device=DEV)
    ws = torch.full((ml.mlora_moe_sort_workspace_bytes(n, E),), 0xA5, dtype=torch.uint8,
                    device=DEV)
    ml.mlora_moe_sort(ids, E, off, order, rows, ws)
    torch.cuda.synchronize()
    return off, order, rows


def _check_sort(ml, host, E):
    got = _sort(ml, torch.from_numpy(host).to(DEV), E)
    for name, g, w in zip(("offsets", "sorted_ids", "slot_rows"), got,
                          moe.sort_by_expert(host, E)):
        assert np.array_equal(_np(g), w), name


@pytest.mark.parametrize("n,experts", [
    (1, 1), (1, 128), (2, 3), (63, 5), (64, 5), (65, 5), (640, 128), (1000, 1024), (1024, 7),
    (1025, 255), (4095, 1), (4096, 127), (4097, 128), (5000, 1023), (8192, 64), (32768, 128),
    (9001, 1024), (40959, 200), (40960, 3), (40961, 200),
    (70001, 1024), (131064, 255)])
def test_sort(ml, n, experts):
    rng = np.random.default_rng(n + experts)
    ids = rng.integers(0, experts, size=n).astype(np.int32)
    ids[rng.random(n) < 0.15] = -1
    ids[rng.random(n) < 0.02] = experts          # past the last one
    ids[rng.random(n) < 0.01] = np.iinfo(np.int32).min
    _check_sort(ml, ids, experts)


@pytest.mark.parametrize("n", [1, 700, 4096, 9000])
def test_sort_one_sided(ml, n):
    for fill in (-1, 0, 9, 10):  # all dropped, all in the first, the last, past it
        _check_sort(ml, np.full(n, fill, dtype=np.int32), 10)
    _check_sort(ml, np.sort(np.arange(n, dtype=np.int32) % 10), 10)
    _check_sort(ml, (np.arange(n, dtype=np.int32) % 10)[::-1].copy(), 10)


def test_sort_ids_from_any_start(ml):
    """ids that start on 4 bytes only."""
    rng = np.random.default_rng(22)
    for n in (700, 5003):
        ids = rng.integers(-1, 33, size=n + 3).astype(np.int32)
        dev = torch.from_numpy(ids).to(DEV)
        for lead in (1, 2, 3):
            got = _sort(ml, dev[lead:lead + n], 33)
            for g, w in zip(got, moe.sort_by_expert(ids[lead:lead + n], 33)):
                assert np.array_equal(_np(g), w)


def test_sort_many_tiles_per_block(ml):
    """More ids than the most blocks hold in one tile each."""
    rng = np.random.default_rng(21)
    n, E = 256 * 4096 + 12345, 40
    ids = rng.integers(-1, E, size=n).astype(np.int32)
    off, order, rows = (_np(t) for t in _sort(ml, torch.from_numpy(ids).to(DEV), E))
    key = np.where(ids < 0, E, ids)
    want = np.argsort(key, kind="stable").astype(np.int32)
    live = int((ids >= 0).sum())
    assert np.array_equal(off, np.searchsorted(key[want], np.arange(E + 1)).astype(np.int32))
    assert np.array_equal(order[:live], want[:live]) and (order[live:] == -1).all()
    back = np.full(n, -1, dtype=np.int32)
    back[want[:live]] = np.arange(live)
    assert np.array_equal(rows, back)


# ---------------------------------------------------------------------------
# dispatch, combine
# ---------------------------------------------------------------------------

SHAPES = [  # tokens, top_k, experts, dim, dropped
    (1, 1, 4, 1, 0.0), (1, 8, 16, 8, 0.0), (3, 2, 4, 7, 0.3), (5, 9, 12, 24, 0.2),
    (80, 8, 128, 2048, 0.1), (33, 4, 20, 512, 0.0), (17, 6, 60, 520, 0.05), (9, 17, 40, 1000, 0.5),
    (12, 3, 8, 4088, 0.0), (6, 2, 9, 1025, 0.4), (7, 5, 5, 8200, 0.1), (300, 2, 64, 64, 1.0)]


def _maps(ml, tokens, k, experts, dropped, seed):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(experts)[:k] if k <= experts else
                    rng.integers(0, experts, k) for _ in range(tokens)]).astype(np.int32)
    ids[rng.random(ids.shape) < dropped] = -1
    if tokens > 2:
        ids[1] = -1                                # a token with no expert at all
    flat = ids.reshape(-1)
    return flat, _sort(ml, torch.from_numpy(flat).to(DEV), experts)


def _rows(shape, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,k,experts,dim,dropped", SHAPES)
def test_dispatch(ml, dtype, tokens, k, experts, dim, dropped):
    flat, (_, order, slots) = _maps(ml, tokens, k, experts, dropped, 31)
    x = _rows((tokens, dim), dtype, 32)
    out = torch.full((tokens * k, dim), 9.0, dtype=x.dtype, device=DEV)
    ml.mlora_moe_dispatch(x, out, order, slots, k)
    assert np.array_equal(_np(out), moe.dispatch(_np(x), _np(order), k))
    # strided rows, an odd column start: the same values, nothing beside them
    wide = torch.full((tokens * k, dim + 9), 5.0, dtype=x.dtype, device=DEV)
    src = torch.zeros((tokens, dim + 3), dtype=x.dtype, device=DEV)
    src[:, 1:dim + 1] = x
    ml.mlora_moe_dispatch(src[:, 1:dim + 1], wide[:, 4:dim + 4], order, slots, k)
    assert torch.equal(wide[:, 4:dim + 4], out)
    assert bool((wide[:, :4] == 5).all()) and bool((wide[:, dim + 4:] == 5).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("by_slot", [False, True])
@pytest.mark.parametrize("tokens,k,experts,dim,dropped", SHAPES)
def test_combine_and_gradient(ml, dtype, by_slot, tokens, k, experts, dim, dropped):
    flat, (_, order, slots) = _maps(ml, tokens, k, experts, dropped, 41)
    rows = _rows((tokens * k, dim), dtype, 42)
    w = torch.softmax(_rows((tokens, k), "f32", 43), 1)
    g = _rows((tokens, dim), dtype, 44)
    half = HALF[rows.dtype]
    if by_slot:
        slots = order = None
    else:
        rows[_np(order) < 0] = float("nan")        # rows no slot names are not read
    clean = torch.nan_to_num(rows)
    hs = None if by_slot else _np(slots)
    for wt in (w, None):
        hw = None if wt is None else _np(wt)
        out = torch.full((tokens, dim), 9.0, dtype=rows.dtype, device=DEV)
        ml.mlora_moe_combine(rows, out, k, wt, slots)
        ref, mag = moe.combine(_np(clean), tokens, k, hw, hs)
        _close(_np(out), ref, mag * (k + 1) * U, half, "out")
        d_rows = torch.full_like(rows, 9.0)
        d_w = torch.full((tokens, k), 9.0, device=DEV)
        ml.mlora_moe_combine_backward(g, rows, wt, d_rows, d_w, k, slots, order)
        r_ref, w_ref, w_mag = moe.combine_gradient(_np(g), _np(clean), k, hw, hs)
        _close(_np(d_rows), r_ref, np.abs(r_ref) * U, half, "d_rows")
        _close(_np(d_w), w_ref, w_mag * (dim / 64 + 24) * U, 0.0, "d_weights")
        again = torch.full_like(rows, 7.0)
        ml.mlora_moe_combine_backward(g, None, wt, again, None, k, slots, order)
        assert torch.equal(again, d_rows)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_combine_strides(ml, dtype):
    tokens, k, experts, dim = 20, 4, 16, 136
    _, (_, order, slots) = _maps(ml, tokens, k, experts, 0.2, 51)
    w = torch.rand((tokens, k), device=DEV)
    rows, g = _rows((tokens * k, dim), dtype, 52), _rows((tokens, dim), dtype, 53)
    out, d_rows = torch.empty_like(g), torch.empty_like(rows)
    d_w = torch.empty_like(w)
    ml.mlora_moe_combine(rows, out, k, w, slots)
    ml.mlora_moe_combine_backward(g, rows, w, d_rows, d_w, k, slots, order)
    for lead in (0, 8, 3):
        def pad(t):
            p = torch.full((t.shape[0], dim + 24), 5.0, dtype=t.dtype, device=DEV)
            p[:, lead:lead + dim] = t
            return p, p[:, lead:lead + dim]
        (_, r2), (_, g2) = pad(rows), pad(g)
        (ob, o2), (db, d2) = pad(torch.zeros_like(g)), pad(torch.zeros_like(rows))
        w2 = torch.empty_like(w)
        ml.mlora_moe_combine(r2, o2, k, w, slots)
        ml.mlora_moe_combine_backward(g2, r2, w, d2, w2, k, slots, order)
        assert torch.equal(o2, out) and torch.equal(d2, d_rows)
        for b in (ob, db):
            assert bool((b[:, :lead] == 5).all()) and bool((b[:, lead + dim:] == 5).all())
        _, w_ref, w_mag = moe.combine_gradient(_np(g), _np(rows), k, _np(w), _np(slots))
        _close(_np(w2), w_ref, w_mag * (dim / 64 + 24) * U, 0.0, "d_weights")


def test_dispatch_gradient_is_the_unweighted_combine(ml):
    """<dispatch(x), g> differentiated by x is combine(g) with unit weights."""
    tokens, k, experts, dim = 13, 4, 10, 72
    _, (_, order, slots) = _maps(ml, tokens, k, experts, 0.2, 61)
    g = _rows((tokens * k, dim), "f32", 62)
    dx = torch.empty((tokens, dim), device=DEV)
    ml.mlora_moe_combine(g, dx, k, None, slots)
    ref = np.zeros((tokens, dim))
    for r, i in enumerate(_np(order)):
        if i >= 0:
            ref[i // k] += _np(g)[r]
    _close(_np(dx), ref, np.abs(ref) * U + 16 * U * k, 0.0, "dx")


def test_combine_reads_rows_past_32_bit_offsets(ml):
    """Rows that start beyond 2^32 elements (and 2^33 bytes)."""
    dim, n_rows = 4096, (1 << 20) + 8
    rows = torch.empty((n_rows, dim), dtype=torch.bfloat16, device=DEV)
    far = torch.tensor([n_rows - 1, 5, n_rows - 3, 0], dtype=torch.int32, device=DEV)
    for r in far.tolist():
        rows[r] = _rows((dim,), "bf16", r % 97)
    out = torch.empty((2, dim), dtype=torch.bfloat16, device=DEV)
    ml.mlora_moe_combine(rows, out, 2, None, far)
    pick = rows[far.long()].float().view(2, 2, dim).sum(1).to(torch.bfloat16)
    assert torch.equal(out, pick)


def test_combine_bad_slot_rows_are_left_out(ml):
    rows = _rows((6, 40), "f32", 71)
    slots = torch.tensor([0, 6, -5, 5, 1 << 30, 2], dtype=torch.int32, device=DEV)
    out = torch.empty((3, 40), device=DEV)
    ml.mlora_moe_combine(rows, out, 2, None, slots)
    assert torch.equal(out, torch.stack([rows[0], rows[5], rows[2]]))


def test_graph_replay_and_other_stream(ml):
    """Router, sort, dispatch, combine and the gradients captured once; every
    replay, after the logits were rewritten in place, equals the eager calls."""
    tokens, k, E, dim = 700, 8, 64, 256
    lg, x = _rows((tokens, E), "bf16", 81), _rows((tokens, dim), "bf16", 82)
    g = _rows((tokens, dim), "bf16", 83)
    n = tokens * k

    def buffers():
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
        return dict(idx=i32(tokens, k), w=torch.zeros((tokens, k), device=DEV), off=i32(E + 1),
                    order=i32(n), slots=i32(n),
                    rows=torch.zeros((n, dim), dtype=x.dtype, device=DEV),
                    out=torch.zeros_like(x), d_rows=torch.zeros((n, dim), dtype=x.dtype, device=DEV),
                    d_w=torch.zeros((tokens, k), device=DEV), d_l=torch.zeros_like(lg),
                    ws=torch.zeros(ml.mlora_moe_sort_workspace_bytes(n, E), dtype=torch.uint8,
                                   device=DEV))

    def step(b):
        ml.mlora_router_topk(lg, b["idx"], b["w"], renormalize=True)
        ml.mlora_moe_sort(b["idx"].view(-1), E, b["off"], b["order"], b["slots"], b["ws"])
        ml.mlora_moe_dispatch(x, b["rows"], b["order"], b["slots"], k)
        ml.mlora_moe_combine(b["rows"], b["out"], k, b["w"], b["slots"])
        ml.mlora_moe_combine_backward(g, b["rows"], b["w"], b["d_rows"], b["d_w"], k, b["slots"],
                                      b["order"])
        ml.mlora_router_topk_backward(lg, b["idx"], b["d_w"], b["d_l"], renormalize=True)

    cap = buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step(cap)
    torch.cuda.current_stream().wait_stream(side)
    for r in range(4):
        lg.copy_(_rows((tokens, E), "bf16", 90 + r))
        eager = buffers()
        step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in eager:
            if name != "ws":
                assert torch.equal(eager[name], cap[name]), (r, name)


def test_binding_refuses(ml):
    lg = torch.randn((4, 16), device=DEV)
    idx = torch.empty((4, 2), dtype=torch.int32, device=DEV)
    w = torch.empty((4, 2), device=DEV)
    for call in (
            lambda: ml.mlora_router_topk(lg.cpu(), idx, w),
            lambda: ml.mlora_router_topk(lg.t(), idx, w),
            lambda: ml.mlora_router_topk(lg, idx[:3], w),
            lambda: ml.mlora_router_topk(lg, idx.t().contiguous().t(), w),
            lambda: ml.mlora_router_topk_backward(lg, idx, w, lg[:, :8]),
            lambda: ml.mlora_moe_sort(idx.view(-1), 16, idx, idx.view(-1), idx.view(-1)),
            lambda: ml.mlora_moe_dispatch(lg, lg, idx.view(-1), idx.view(-1), 2),
            lambda: ml.mlora_moe_combine(lg, lg[:, :8], 1),
            lambda: ml.mlora_moe_combine(lg, lg[:2], 2, w)):
        with pytest.raises(ValueError):
            call()
    for call in (
            lambda: ml.mlora_router_topk(lg.half(), idx, w),
            lambda: ml.mlora_router_topk(lg, idx.long(), w),
            lambda: ml.mlora_router_topk(lg, idx, w.bfloat16()),
            lambda: ml.mlora_moe_combine(lg, lg.bfloat16(), 1)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ml.MloraError):
        ml.mlora_router_topk(lg[:, :1], idx, w)  # top_k above the experts
