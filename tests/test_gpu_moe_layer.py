"""GPU test of the example MoE layer (examples/moe_layer.py) against plain fp64:
a decode step with adapters, captured in a graph too, and a training step.

Tolerance of the decode step: gate/up and down are each rounded to bf16 twice
(product, fold), the activation once, the output once; a rounding is at most
2^-8 of its value, and the sums behind it average the errors of their terms, so
six of them bound the relative L2: 6 x 2^-8. The training step is fp32: sums of
at most a few hundred products in the rows' order, 2^-24 x 300 of the values'
absolute sums."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest

from oracle import moe
from tests.common import rel_l2

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_layer
    return moe_layer


def _np(t):
    return t.detach().double().cpu().numpy()


def _reference(router, made, x, indices, row_adapter, group=64):
    xs, idx = _np(x), indices.cpu().numpy()
    weights = {}
    for name, (q, s, a, b) in made.items():
        w = moe.w4_weights(q.cpu().numpy(), _np(s), None, q.shape[2] * 2, group)
        weights[name] = (w, w + 0.5 * _np(b) @ _np(a))
    logits = xs @ _np(router).T
    w = moe.router_weights(logits, idx, True)
    out = np.zeros_like(xs)
    for t in range(xs.shape[0]):
        on = int(row_adapter[t] >= 0)
        for j, e in enumerate(idx[t]):
            gate, up = weights["gate"][on][e] @ xs[t], weights["up"][on][e] @ xs[t]
            out[t] += w[t, j] * (weights["down"][on][e] @ (gate / (1 + np.exp(-gate)) * up))
    return out


def test_decode_step(example):
    layer, router, made = example.example_layer()
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((24, router.shape[1]), generator=g, device="cuda").to(torch.bfloat16)
    host_map = np.array([0] * 20 + [-1] * 4, dtype=np.int32)
    row_adapter = torch.from_numpy(host_map).cuda()
    out = layer(x, row_adapter).clone()
    ref = _reference(router, made, x, layer.indices[:24], host_map)
    rel = rel_l2(_np(out), ref)
    print(f"decode step rel_l2={rel:.3e}", flush=True)
    assert rel <= 6 * 2.0 ** -8
    # the choice itself, by the bf16 logits that the layer saw
    assert np.array_equal(layer.indices[:24].cpu().numpy(),
                          moe.router_choice(_np(x @ router.t()), 4))
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, row_adapter)
        with torch.cuda.graph(graph, stream=side):
            captured = layer(x, row_adapter)
    torch.cuda.current_stream().wait_stream(side)
    for r in range(3):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        eager = layer(x, row_adapter).clone()
        torch.cuda.synchronize()
        captured.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, eager), r


def test_train_step(example):
    g = torch.Generator(device="cuda").manual_seed(4)
    t, dim, E, k = 50, 72, 12, 3
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, logits, d_out, gain = rnd(t, dim), rnd(t, E), rnd(t, dim), rnd(E) + 2

    def experts(rows, offsets):
        of = torch.repeat_interleave(gain, (offsets[1:] - offsets[:-1]).long()).unsqueeze(1)
        return rows * of, lambda d_rows: d_rows * of

    out, grads = example.train_step(x, logits, d_out, k, experts)
    lg, xs, dh, gn = _np(logits), _np(x), _np(d_out), _np(gain)
    idx = moe.router_choice(lg, k)
    w = moe.router_weights(lg, idx, True)
    scale = (w * gn[idx]).sum(1, keepdims=True)
    mag = (w * np.abs(gn[idx])).sum(1, keepdims=True)
    tol = 300 * 2.0 ** -24
    assert (np.abs(_np(out) - xs * scale) <= tol * mag * np.abs(xs) + 1e-30).all()
    assert (np.abs(_np(grads["x"]) - dh * scale) <= tol * mag * np.abs(dh) + 1e-30).all()
    dots = (dh * xs).sum(1, keepdims=True)
    d_w = gn[idx] * dots
    w_mag = np.abs(gn[idx]) * (np.abs(dh) * np.abs(xs)).sum(1, keepdims=True)
    assert (np.abs(_np(grads["weights"]) - d_w) <= tol * w_mag).all()
    ref = moe.router_gradient(lg, idx, d_w, True)
    bound = tol * 2 * w_mag.max(1, keepdims=True)
    assert (np.abs(_np(grads["logits"]) - ref) <= bound).all()
    order = np.argsort(idx.reshape(-1), kind="stable")
    d_rows = (w[..., None] * dh[:, None]).reshape(-1, dim)[order]
    assert (np.abs(_np(grads["rows"]) - d_rows) <= tol * np.abs(d_rows) + 1e-30).all()


def test_main_runs(example, capsys):
    example.main()
    assert "training step" in capsys.readouterr().out
