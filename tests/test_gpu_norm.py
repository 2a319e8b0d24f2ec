"""GPU tests of the norms around a block and their gradients."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8  # noqa: E402
from tests.fp8_cases import F32, U, close, to64  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
KW = dict(residual_scale=0.75, y_scale=1.5, eps=1e-5)


@pytest.fixture(scope="module")
def ml():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_lora_amd
    return moe_expert_lora_amd


def strided(t, extra):
    wide = torch.zeros((t.shape[0], t.shape[1] + extra), dtype=t.dtype, device=DEV)
    return (wide[:, extra // 2:extra // 2 + t.shape[1]] if extra else wide).copy_(t)


def inputs(seed, T, D, dtype, y=True, post=True, gate="none", w="f32", extra=0):
    rng = np.random.default_rng(seed)
    mat = lambda std: strided(torch.from_numpy(rng.normal(0, std, (T, D))).to(  # noqa: E731
        DEV, TORCH[dtype]), extra)
    vec = lambda: torch.from_numpy(rng.normal(1, 0.2, D)).to(DEV, TORCH[w])  # noqa: E731
    d = dict(residual=mat(2.0), y=mat(1.0) if y else None, x_weight=vec(),
             y_weight=vec() if y and post else None, gate=None)
    if y and gate == "channel":
        d["gate"] = torch.from_numpy(rng.normal(0, 1, D)).to(DEV, TORCH[dtype])
    elif y and gate == "token":
        d["gate"] = torch.from_numpy(rng.normal(0, 1, (T, 1))).to(DEV, TORCH[dtype])
    elif y and gate == "full":
        d["gate"] = mat(1.0)
    return d, (mat(1.0), mat(1.0))


def in64(d):
    return {k: None if v is None else to64(v) for k, v in d.items()}


def absolute(d, offset):
    """The magnitudes that errors of the single steps are relative to: the parts of r
    and, through its norm, of x. A sum's roundings and a norm's are below 64 units of
    2^-24 each for up to 16384 values (16 a thread, then a tree)."""
    a = in64(d)
    f = lambda v: None if v is None else np.abs(v)  # noqa: E731
    n = a["y"]
    if n is not None and a["y_weight"] is not None:
        n = n / np.sqrt((n * n).mean(1, keepdims=True) + KW["eps"]) * (a["y_weight"] + offset)
    parts = KW["residual_scale"] * np.abs(a["residual"])
    if n is not None:
        parts = parts + KW["y_scale"] * np.abs(1.0 if a["gate"] is None else a["gate"]) * np.abs(n)
    r, _ = fp8.block_norm(**a, **KW, offset=offset)
    R = 1 / np.sqrt((r * r).mean(1, keepdims=True) + KW["eps"])
    # how much the parts' errors can move the row's norm
    spread = (np.abs(r) * parts).mean(1, keepdims=True) * R * R + 1
    return parts, R, spread, f(n)


STEP = 64 * F32


def check_forward(ml, d, dtype, offset=0.0, **out):
    ml.mlora_block_norm(d["residual"], y=d["y"], x_weight=d["x_weight"], y_weight=d["y_weight"],
                        gate=d["gate"], weight_offset=offset, **KW, **out)


def run_forward(ml, d, dtype, offset=0.0):
    want_r, want_x = fp8.block_norm(**in64(d), **KW, offset=offset)
    parts, R, spread, _ = absolute(d, offset)
    r, x = torch.empty_like(d["residual"]), torch.empty_like(d["residual"])
    check_forward(ml, d, dtype, offset, r=r, x=x)
    err = parts * STEP
    close(to64(r), want_r, err + (np.abs(want_r) + err) * U[dtype])
    w = 1.0 if d["x_weight"] is None else np.abs(to64(d["x_weight"]) + offset)
    err = (parts + np.abs(want_r) * spread) * R * w * STEP
    close(to64(x), want_x, err + (np.abs(want_x) + err) * U[dtype])


def outputs(ml, d, want):
    T, D = d["residual"].shape
    o = {"d_residual": torch.empty_like(d["residual"]), "d_x_weight": torch.empty(D, device=DEV)}
    if d["y"] is not None:
        o["d_y"] = torch.empty_like(d["y"])
    if d["y_weight"] is not None:
        o["d_y_weight"] = torch.empty(D, device=DEV)
    if d["gate"] is not None:
        full = d["gate"].dim() == 2 and d["gate"].shape[1] == D and D > 1
        o["d_gate"] = torch.empty_like(d["gate"]) if full else torch.empty(
            d["gate"].shape, device=DEV)
    return o


def backward(ml, d, d_r, d_x, o, offset=0.0, **kw):
    T, D = d["residual"].shape
    ws = torch.full((ml.mlora_block_norm_backward_workspace_bytes(T, D),), 0xff, dtype=torch.uint8,
                    device=DEV)
    ml.mlora_block_norm_backward(d["residual"], d_r=d_r, d_x=d_x, y=d["y"],
                                 x_weight=d["x_weight"], y_weight=d["y_weight"], gate=d["gate"],
                                 weight_offset=offset, workspace=ws, **KW, **o, **kw)


def run_backward(ml, d, grads, dtype, offset=0.0, use=(True, True)):
    d_r, d_x = (g if u else None for g, u in zip(grads, use))
    T, D = d["residual"].shape
    o = outputs(ml, d, None)
    backward(ml, d, d_r, d_x, o, offset)
    zero = np.zeros((T, D))
    gr, gx = (zero if g is None else to64(g) for g in (d_r, d_x))
    a = in64(d)
    want = fp8.block_norm_gradient(d_r=gr, d_x=gx, **a, **KW, offset=offset)
    # magnitudes, step by step as in the definition
    parts, R, spread, n = absolute(d, offset)
    r, _ = fp8.block_norm(**a, **KW, offset=offset)
    wx = 1.0 if a["x_weight"] is None else np.abs(a["x_weight"] + offset)
    h = (parts + np.abs(r) * spread) * R
    g = np.abs(gx) * wx
    m = np.abs(gr) + R * spread * (g + h * (g * h).mean(1, keepdims=True))
    mags = {"residual": KW["residual_scale"] * m, "x_weight": (np.abs(gx) * h).sum(0)}
    if a["y"] is not None:
        gt = 1.0 if a["gate"] is None else np.abs(a["gate"])
        d_n = KW["y_scale"] * m * gt
        mags["y"] = d_n
        if a["y_weight"] is not None:
            Ry = 1 / np.sqrt((a["y"] ** 2).mean(1, keepdims=True) + KW["eps"])
            v = np.abs(a["y"]) * Ry
            u = d_n * np.abs(a["y_weight"] + offset)
            mags["y"] = Ry * (u + v * (u * v).mean(1, keepdims=True))
            mags["y_weight"] = (d_n * v).sum(0)
        if a["gate"] is not None:
            dg = KW["y_scale"] * m * n
            mags["gate"] = dg.sum(0) if a["gate"].ndim == 1 else \
                dg.sum(1, keepdims=True) if a["gate"].shape[1] == 1 and D > 1 else dg
    for name, ref in want.items():
        got = o["d_" + name]
        # five norms or sums over a row, and for sums over the tokens one rounding each
        err = mags[name] * (5 * STEP + (T * F32 if ref.ndim == 1 else 0.0))
        half = U["bf16"] if got.dtype == torch.bfloat16 else U["f32"]
        close(to64(got), ref, err + (np.abs(ref) + err) * half, name)


# tokens, dim: every number of threads a row, both sides of each limit, odd widths
SIZES = [(1, 1), (3, 7), (5, 512), (9, 513), (4, 1024), (2, 1032), (80, 2048), (3, 2056),
         (1, 4096), (6, 4100), (2, 8192), (3, 8193), (2, 16384), (700, 40)]
GATES = ["none", "channel", "token", "full"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", SIZES)
def test_sizes(ml, T, D, dtype):
    gate = GATES[(T + D) % 4]
    d, grads = inputs(D, T, D, dtype, gate=gate)
    run_forward(ml, d, dtype)
    run_backward(ml, d, grads, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("D", [96, 1536])
def test_forms(ml, D, gate, post, dtype):
    d, grads = inputs(3, 2100 if D == 96 else 21, D, dtype, post=post, gate=gate, w="bf16")
    run_forward(ml, d, dtype, offset=1.0)
    run_backward(ml, d, grads, dtype, offset=1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("extra", [3, 16])
def test_strides(ml, extra, dtype):
    d, grads = inputs(4, 19, 640, dtype, gate="full", extra=extra)
    run_forward(ml, d, dtype)
    run_backward(ml, d, grads, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_a_block(ml, dtype):
    """residual alone: the first norm of a model; and no weight."""
    d, grads = inputs(5, 33, 768, dtype, y=False)
    run_forward(ml, d, dtype)
    run_backward(ml, d, grads, dtype)
    d["x_weight"] = None
    run_forward(ml, d, dtype)


@pytest.mark.parametrize("use", [(True, False), (False, True)])
@pytest.mark.parametrize("gate", GATES)
def test_one_gradient_alone(ml, gate, use):
    """Many rows a group of threads, with and without the sums over a row between
    them; d_x alone without a norm of y leaves one sum a row."""
    for post in (False, True):
        d, grads = inputs(6, 3000, 1536, "f32", post=post, gate=gate)
        run_backward(ml, d, grads, "f32", use=use)


def test_outputs_one_by_one(ml):
    d, (d_r, d_x) = inputs(7, 50, 256, "bf16", gate="channel")
    whole = outputs(ml, d, None)
    backward(ml, d, d_r, d_x, whole)
    for name, want in whole.items():
        got = torch.empty_like(want)
        backward(ml, d, d_r, d_x, {name: got})
        assert torch.equal(got, want), name
    r, x = torch.empty_like(d_r), torch.empty_like(d_r)
    check_forward(ml, d, "bf16", r=r, x=x)
    only_r, only_x = torch.empty_like(d_r), torch.empty_like(d_r)
    check_forward(ml, d, "bf16", r=only_r)
    check_forward(ml, d, "bf16", x=only_x)
    assert torch.equal(only_r, r) and torch.equal(only_x, x)


@pytest.mark.parametrize("D", [256, 2048, 5000])
def test_in_place(ml, D):
    d, (d_r, d_x) = inputs(8, 37, D, "bf16", gate="token")
    r, x = torch.empty_like(d_r), torch.empty_like(d_r)
    check_forward(ml, d, "bf16", r=r, x=x)
    o = {"d_residual": torch.empty_like(d_r), "d_y": torch.empty_like(d_r)}
    backward(ml, d, d_r, d_x, o)
    gr, gx = d_r.clone(), d_x.clone()
    backward(ml, d, gr, gx, {"d_residual": gr, "d_y": gx})
    assert torch.equal(gr, o["d_residual"]) and torch.equal(gx, o["d_y"])
    e = {k: None if v is None else v.clone() for k, v in d.items()}
    check_forward(ml, e, "bf16", r=e["residual"], x=e["y"])
    assert torch.equal(e["residual"], r) and torch.equal(e["y"], x)


def test_zero_rows_and_rows_that_are_not_finite(ml):
    d, (d_r, d_x) = inputs(9, 12, 300, "bf16", gate="full")
    r, x = torch.empty_like(d_r), torch.empty_like(d_r)
    check_forward(ml, d, "bf16", r=r, x=x)
    o = {"d_residual": torch.empty_like(d_r), "d_y": torch.empty_like(d_r)}
    backward(ml, d, d_r, d_x, o)
    e = {k: None if v is None else v.clone() for k, v in d.items()}
    e["y"][2, 5], e["residual"][7, 0] = float("nan"), float("inf")
    e["y"][4], e["residual"][4] = 0, 0
    r2, x2 = torch.empty_like(d_r), torch.empty_like(d_r)
    check_forward(ml, e, "bf16", r=r2, x=x2)
    o2 = {"d_residual": torch.empty_like(d_r), "d_y": torch.empty_like(d_r)}
    backward(ml, e, d_r, d_x, o2)
    keep = [i for i in range(12) if i not in (2, 4, 7)]
    for a, b in ((r, r2), (x, x2), (o["d_residual"], o2["d_residual"]), (o["d_y"], o2["d_y"])):
        assert torch.equal(a[keep], b[keep])
    assert (r2[4] == 0).all() and (x2[4] == 0).all()
    assert o2["d_residual"][4].isfinite().all() and o2["d_y"][4].isfinite().all()
    assert x2[2].isnan().all()


def test_no_tokens(ml):
    """Sums over no tokens are zeros."""
    D = 200
    e = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    d = dict(residual=e(0, D), y=e(0, D), x_weight=e(D), y_weight=e(D), gate=e(D))
    check_forward(ml, d, "f32", r=e(0, D), x=e(0, D))
    o = dict(d_x_weight=e(D).fill_(3), d_y_weight=e(D).fill_(3), d_gate=e(D).fill_(3),
             d_residual=e(0, D), d_y=e(0, D))
    backward(ml, d, e(0, D), e(0, D), o)
    assert all((o[k] == 0).all() for k in ("d_x_weight", "d_y_weight", "d_gate"))


@pytest.mark.parametrize("D", [256, 2048])
def test_streams_graphs_and_reruns(ml, D):
    d, (d_r, d_x) = inputs(10, 2500, D, "bf16", gate="channel")
    r, x = torch.empty_like(d_r), torch.empty_like(d_r)
    o = outputs(ml, d, None)
    ws = torch.empty(ml.mlora_block_norm_backward_workspace_bytes(2500, D), dtype=torch.uint8,
                     device=DEV)
    kw = dict(y=d["y"], x_weight=d["x_weight"], y_weight=d["y_weight"], gate=d["gate"], **KW)

    def step(stream=None):
        ml.mlora_block_norm(d["residual"], r=r, x=x, stream=stream, **kw)
        ml.mlora_block_norm_backward(d["residual"], d_r=d_r, d_x=d_x, workspace=ws, stream=stream,
                                     **o, **kw)
        return [t.clone() for t in (r, x, *o.values())] if stream is None else None

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, (r, x, *o.values())))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ml.mlora_block_norm(d["residual"], r=r, x=x, **kw)
        ml.mlora_block_norm_backward(d["residual"], d_r=d_r, d_x=d_x, workspace=ws, **o, **kw)
    for i in range(4):
        d["y"].copy_(torch.randn_like(d_r))
        d_x.copy_(torch.randn_like(d_r))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (r, x, *o.values())]
        assert all(torch.equal(a, b) for a, b in zip(got, step())), i


def test_python_refuses(ml):
    d, (d_r, d_x) = inputs(11, 4, 64, "f32", gate="full")
    res, y, r = d["residual"], d["y"], torch.empty_like(d_r)
    gate1 = torch.ones(64, device=DEV)
    for error, call in [
            (TypeError, lambda: ml.mlora_block_norm(res, r=r.bfloat16())),
            (ValueError, lambda: ml.mlora_block_norm(res, r=r[:3])),
            (TypeError, lambda: ml.mlora_block_norm(res, r=r, y=y.bfloat16())),
            (ValueError, lambda: ml.mlora_block_norm(res, r=r, x_weight=gate1[:63])),
            (TypeError, lambda: ml.mlora_block_norm(res, r=r, x=y, y=y, x_weight=gate1,
                                                    y_weight=gate1.bfloat16())),
            (ValueError, lambda: ml.mlora_block_norm(res, r=r, y=y, gate=gate1[:63])),
            (ValueError, lambda: ml.mlora_block_norm(res, r=r, y=y, gate=y[:3])),
            (TypeError, lambda: ml.mlora_block_norm(res, r=r, y=y, gate=gate1.bfloat16())),
            (ml.MloraError, lambda: ml.mlora_block_norm(res)),
            (ml.MloraError, lambda: ml.mlora_block_norm(res, r=r, x=r)),
            (ml.MloraError, lambda: ml.mlora_block_norm(res, r=r, gate=gate1)),
            (ml.MloraError, lambda: ml.mlora_block_norm(res, r=r, eps=-1.0)),
            (ValueError, lambda: ml.mlora_block_norm(res.cpu(), r=r)),
            (ml.MloraError, lambda: ml.mlora_block_norm_backward(res, d_residual=r)),
            (ml.MloraError, lambda: ml.mlora_block_norm_backward(res, d_x=d_x, d_x_weight=gate1)),
            (ml.MloraError, lambda: ml.mlora_block_norm_backward(res, d_x=d_x, d_y=r)),
            (ValueError, lambda: ml.mlora_block_norm_backward(res, d_x=d_x, d_gate=gate1)),
            (TypeError, lambda: ml.mlora_block_norm_backward(
                res, d_x=d_x, y=y, gate=gate1, d_gate=gate1.bfloat16())),
            (ValueError, lambda: ml.mlora_block_norm_backward(
                res, d_x=d_x, y=y, gate=gate1, d_gate=gate1[:5]))]:
        with pytest.raises(error):
            call()
