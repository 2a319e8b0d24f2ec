"""GPU tests of how the 8-bit products, the layer of a few tokens and the norms
around a block are used together and at their limits: graphs that share a
workspace, calls on two streams at once, offsets past 32 bits, the largest lists
of experts, more rows than workgroups for wide rows."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8  # noqa: E402
from tests import test_gpu_few_tokens as few  # noqa: E402
from tests import test_gpu_norm as norm  # noqa: E402
from tests.fp8_cases import close, product_error, to64, weights  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def ml():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_lora_amd
    return moe_expert_lora_amd


def _graph(run):
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        with torch.cuda.graph(graph, stream=side):
            run()
    torch.cuda.current_stream().wait_stream(side)
    return graph


def test_layers_of_two_graphs_share_a_workspace(ml):
    sizes = [(16, 40, 6, 700, 300), (3, 12, 2, 1024, 520)]
    cases = [few.Case(ml, 20 + i, *s, "bf16") for i, s in enumerate(sizes)]
    ws = max((c.ws for c in cases), key=torch.numel)
    want = []
    for c in cases:
        c.check()  # with a workspace of its own
        want.append(c.out.clone())
        c.ws = ws
    graphs = [_graph(c.run) for c in cases]
    for i in range(6):
        c, graph = cases[i % 2], graphs[i % 2]
        c.out.zero_()
        graph.replay()
        if i == 3:
            cases[1 - i % 2].run()  # an eager call between them
        torch.cuda.synchronize()
        assert torch.equal(c.out, want[i % 2]), i


def _norm_call(ml, seed, T, D, gate, dtype):
    d, (d_r, d_x) = norm.inputs(seed, T, D, dtype, gate=gate)
    r, x = torch.empty_like(d_r), torch.empty_like(d_r)
    o = norm.outputs(ml, d, None)
    ws = torch.empty(ml.mlora_block_norm_backward_workspace_bytes(T, D), dtype=torch.uint8,
                     device=DEV)

    def run(ws=ws, stream=None):
        kw = dict(y=d["y"], x_weight=d["x_weight"], y_weight=d["y_weight"], gate=d["gate"],
                  stream=stream, **norm.KW)
        ml.mlora_block_norm(d["residual"], r=r, x=x, **kw)
        ml.mlora_block_norm_backward(d["residual"], d_r=d_r, d_x=d_x, workspace=ws, **o, **kw)

    return run, [r, x, *o.values()], ws


def test_norms_of_two_graphs_share_a_workspace(ml):
    calls = [_norm_call(ml, 1, 900, 1000, "channel", "bf16"),
             _norm_call(ml, 2, 333, 2048, "token", "f32")]
    shared = max((c[2] for c in calls), key=torch.numel)
    want = []
    for run, outs, _ in calls:
        run()
        want.append([t.clone() for t in outs])
    graphs = [_graph(lambda run=run: run(shared)) for run, _, _ in calls]
    for i in range(6):
        for t in calls[i % 2][1]:
            t.zero_()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(calls[i % 2][1], want[i % 2])), i


def test_two_streams_at_once(ml):
    """Everything on two streams at the same time, workspaces of their own."""
    sets = []
    for i in range(2):
        layer = few.Case(ml, 30 + i, 16, 32, 4, 512, 384, "bf16")
        run_norm, outs, _ = _norm_call(ml, 40 + i, 2000, 512, "channel", "bf16")
        rng = np.random.default_rng(50 + i)
        w, s = weights(rng, 4, 300, 520)
        route = ml.make_fp8_route(torch.from_numpy(w).to(DEV), torch.from_numpy(s).to(DEV))
        x = torch.randn((900, 520), device=DEV).bfloat16()
        q = torch.empty((900, ml.mlora_fp8_row_width(520)), dtype=torch.uint8, device=DEV)
        qs, y = torch.empty((5, 900), device=DEV), torch.empty((900, 300), device=DEV)
        off = torch.tensor([0, 100, 100, 700, 900], dtype=torch.int32, device=DEV)

        def run(stream=None, layer=layer, run_norm=run_norm, route=route, x=x, q=q, qs=qs, y=y,
                off=off):
            layer.run(stream=stream)
            run_norm(stream=stream)
            ml.mlora_fp8_quant(x, q, qs, stream=stream)
            ml.mlora_fp8_gemm(route, q, qs, y, off, stream=stream)

        sets.append((run, [layer.out, y, *outs]))
    want = []
    for run, outs in sets:
        run()
        want.append([t.clone() for t in outs])
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for (_, outs), s in zip(sets, streams):
            for t in outs:
                t.zero_()
            s.wait_stream(torch.cuda.current_stream())
        for (run, _), s in zip(sets, streams):
            run(s)
        torch.cuda.synchronize()
        for (_, outs), w in zip(sets, want):
            assert all(torch.equal(a, b) for a, b in zip(outs, w))


@pytest.mark.parametrize("n", [40, 32000])  # rows straight from memory, large tiles
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(ml, n, dtype):
    """q of almost 4 GiB, rows and results of more than 2^31 elements between their
    first and last row: those of rows next to each other, bit for bit."""
    rng = np.random.default_rng(n)
    K, N, out_ld = 200, 136, (1 << 31) // n + 4096
    width, q_ld = ml.mlora_fp8_row_width(K), ((1 << 32) - 512) // n // 16 * 16
    w, s = weights(rng, 1, N, K)
    route = ml.make_fp8_route(torch.from_numpy(w).to(DEV), torch.from_numpy(s).to(DEV))
    t = few.TORCH[dtype]
    x = torch.randn((n, K), device=DEV).to(t)
    far_x = torch.empty((n, out_ld), dtype=t, device=DEV)[:, :K]
    far_x.copy_(x)
    q = torch.empty((n, width), dtype=torch.uint8, device=DEV)
    far_q = torch.empty((n, q_ld), dtype=torch.uint8, device=DEV)[:, :width]
    qs, far_qs = (torch.empty((2, n), device=DEV) for _ in range(2))
    ml.mlora_fp8_quant(x, q, qs)
    ml.mlora_fp8_quant(far_x, far_q, far_qs)
    written = slice(0, -(-K // 128) * 128)
    assert torch.equal(q[:, written], far_q[:, written]) and torch.equal(qs, far_qs)
    out = torch.empty((n, N), dtype=t, device=DEV)
    far = torch.empty((n, out_ld), dtype=t, device=DEV)[:, :N]
    ml.mlora_fp8_gemm(route, q, qs, out)
    ml.mlora_fp8_gemm(route, far_q, far_qs, far)
    assert torch.equal(out, far)
    last = slice(n - 3, n)
    rows = fp8.rows_of(q[last].cpu().numpy(), qs[:, last].cpu().numpy(), K)
    full = fp8.expand(w, s)[0]
    ref = rows @ full.T
    close(to64(far[last]), ref, product_error(ref, np.abs(rows) @ np.abs(full).T, K, dtype))
    del far_q, far_x, far
    torch.cuda.empty_cache()


def test_norm_offsets_past_32_bits(ml):
    T, D = 40, 300
    d, grads = norm.inputs(3, T, D, "bf16", gate="full")
    near = [d["residual"], d["y"], d["gate"], *grads]
    far = [torch.empty((T, (1 << 31) // T + 64), dtype=torch.bfloat16, device=DEV)[:, :D]
           for _ in range(6)]
    for a, b in zip(near, far):
        b.copy_(a)
    kw = dict(x_weight=d["x_weight"], y_weight=d["y_weight"], **norm.KW)
    x, d_y = torch.empty_like(near[0]), torch.empty_like(near[0])
    ml.mlora_block_norm(near[0], x=x, y=near[1], gate=near[2], **kw)
    ml.mlora_block_norm(far[0], x=far[5], y=far[1], gate=far[2], **kw)
    assert torch.equal(x, far[5])
    ml.mlora_block_norm_backward(near[0], d_r=near[3], d_x=near[4], d_y=d_y, y=near[1],
                                 gate=near[2], **kw)
    ml.mlora_block_norm_backward(far[0], d_r=far[3], d_x=far[4], d_y=far[5], y=far[1],
                                 gate=far[2], **kw)
    assert torch.equal(d_y, far[5])
    del far
    torch.cuda.empty_cache()


# tokens, experts, top_k, dim, hidden: every expert, the most choices, wide rows whose x
# is read again for each tile
@pytest.mark.parametrize("size", [(16, 1024, 64, 40, 24), (16, 64, 64, 130, 60),
                                  (2, 3, 2, 5000, 70), (2, 3, 2, 70, 9000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_limits(ml, size, dtype):
    few.Case(ml, 60, *size, dtype).check()


# more rows than groups of threads, for each number of threads a row
@pytest.mark.parametrize("T,D", [(5000, 7), (4300, 100), (2100, 1001), (1100, 4095), (600, 5003),
                                 (540, 16381)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_many_rows(ml, T, D, dtype):
    d, grads = norm.inputs(5, T, D, dtype, gate="channel")
    norm.run_forward(ml, d, dtype)
    norm.run_backward(ml, d, grads, dtype)


def test_norm_outputs_are_apart(ml):
    d, (d_r, d_x) = norm.inputs(6, 4, 64, "f32", gate="full")
    o = norm.outputs(ml, d, None)
    with pytest.raises(ml.MloraError, match="same memory"):
        norm.backward(ml, d, d_r, d_x, {**o, "d_y": o["d_residual"]})
