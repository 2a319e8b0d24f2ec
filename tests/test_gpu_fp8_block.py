"""GPU test of the example's 8-bit block (examples/moe_layer.py) against plain fp64
without any rounding of rows: a decode step, a prefill batch with adapters, and
the gradients of a training step.

Tolerances are of relative L2. A value in [1, 2) 2^e has E4M3 neighbours 2^-3 2^e
apart, so a rounding's error has a root mean square of at most Q = 2^-4 / sqrt(3)
of the value, and errors of different k are independent: a product's relative L2
is at most that of its rows. From x, gate and up are off by Q each and alike,
silu(gate) * up by 1.3 Q + Q (|g silu'(g)| has 1.3 times silu's root mean square at
most), its own rounding adds Q: sqrt(2.3^2 + 1) = 2.5 Q, with bf16's roundings
(6 x 2^-8 = 0.65 Q) within 4 Q. Gradients: those of the down product's rows Q, times
silu' and up 2.3 Q, rounded once more Q; the combine weights' 2.5 Q: within 5 Q.
The decode step's rows are not rounded to 8 bits: as in a step of the 4-bit layer
6 x 2^-8, and two norms' outputs 2 x 2^-8."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8, moe  # noqa: E402
from tests.common import rel_l2  # noqa: E402

pytestmark = pytest.mark.gpu

Q = 2.0 ** -4 / 3 ** 0.5
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIZES = [(16, 512, 256, 4), (6, 200, 136, 2)]  # experts, dim, hidden, top_k


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_layer
    return moe_layer


class Case:
    def __init__(self, example, tokens, E, dim, hidden, top_k):
        self.block, made = example.example_block(E, dim, hidden, top_k=top_k)
        g = torch.Generator(device="cuda").manual_seed(7)
        self.residual = torch.randn((tokens, dim), generator=g, device="cuda").to(torch.bfloat16)
        self.d_out = torch.randn((tokens, dim), generator=g, device="cuda").to(torch.bfloat16)
        self.plain, self.adapted = {}, {}
        for name, (w, s, a, b) in made.items():
            self.plain[name] = fp8.expand(w.view(torch.uint8).cpu().numpy(), s.cpu().numpy())
            self.adapted[name] = self.plain[name] + 0.5 * _np(b) @ _np(a)

    def logits(self, residual):
        """What the block's router sees: the choice has to be of these."""
        x = torch.empty_like(residual)
        self.block_norm(residual, x)
        return _np(x @ self.block.router.t())

    def block_norm(self, residual, x):
        import moe_expert_lora_amd as ml
        ml.mlora_block_norm(residual, x=x, x_weight=self.block.norm_in)

    def moe(self, residual, row_adapter):
        b, k = self.block, self.block.top_k
        _, x = fp8.block_norm(_np(residual), x_weight=_np(b.norm_in))
        lg = self.logits(residual)
        idx = moe.router_choice(lg, k)
        w = moe.router_weights(lg, idx, True)
        out = np.zeros_like(x)
        for t in range(x.shape[0]):
            of = self.adapted if row_adapter[t] >= 0 else self.plain
            for j, e in enumerate(idx[t]):
                act = fp8.silu(of["gate"][e] @ x[t]) * (of["up"][e] @ x[t])
                out[t] += w[t, j] * (of["down"][e] @ act)
        return out

    def added(self, residual, row_adapter):
        """What the block adds to the residual."""
        y = self.moe(residual, row_adapter)
        r, _ = fp8.block_norm(np.zeros_like(y), y=y, y_weight=_np(self.block.norm_out))
        return r


@pytest.mark.parametrize("size", SIZES)
def test_prefill(example, size):
    c = Case(example, 150, *size)
    host_map = np.where(np.arange(150) < 90, 0, -1).astype(np.int32)
    out = c.block.prefill(c.residual, torch.from_numpy(host_map).cuda())
    got = _np(out) - _np(c.residual)
    ref = c.added(c.residual, host_map)
    for rows in (slice(0, 90), slice(90, 150)):
        rel = rel_l2(got[rows], ref[rows])
        print(f"prefill rel_l2={rel:.3e}", flush=True)
        assert rel <= 4 * Q
    # the adapters are more than that
    assert rel_l2(c.added(c.residual, host_map * 0 - 1)[:90], ref[:90]) > 8 * Q


@pytest.mark.parametrize("size", SIZES)
def test_decode(example, size):
    c = Case(example, 16, *size)
    for t in (1, 5, 16):
        residual = c.residual[:t]
        got = _np(c.block.decode(residual)) - _np(residual)
        rel = rel_l2(got, c.added(residual, -np.ones(t)))
        print(f"decode of {t} rel_l2={rel:.3e}", flush=True)
        assert rel <= 8 * 2.0 ** -8


def test_prefill_and_decode_agree(example):
    """The same tokens by both ways: within the rounding of the prefill's rows."""
    c = Case(example, 12, *SIZES[0])
    none = torch.full((12,), -1, dtype=torch.int32, device="cuda")
    a = _np(c.block.prefill(c.residual, none)) - _np(c.residual)
    b = _np(c.block.decode(c.residual)) - _np(c.residual)
    assert rel_l2(a, b) <= 4 * Q


def test_captured(example):
    c = Case(example, 9, *SIZES[0])
    x = c.residual
    row_adapter = torch.tensor([0, -1] * 4 + [0], dtype=torch.int32, device="cuda")
    d_out = c.d_out

    def run():
        out, grads = c.block.train(x, d_out)
        return [c.block.prefill(x, row_adapter), c.block.decode(x).clone(), out, *grads.values()]

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        with torch.cuda.graph(graph, stream=side):
            captured = run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.Generator(device="cuda").manual_seed(8)
    for r in range(3):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        eager = [v.clone() for v in run()]
        for v in captured:
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(captured, eager)):
            assert torch.equal(a, b), (r, i)


@pytest.mark.parametrize("size", SIZES)
def test_train(example, size):
    c = Case(example, 96, *size)
    out, grads = c.block.train(c.residual, c.d_out)
    b, k = c.block, c.block.top_k
    idx = torch.from_numpy(moe.router_choice(c.logits(c.residual), k)).long()
    leaf = {n: t.detach().double().cpu().requires_grad_() for n, t in
            (("residual", c.residual), ("norm_in", b.norm_in), ("norm_out", b.norm_out),
             ("router", b.router))}
    W = {n: torch.from_numpy(w) for n, w in c.plain.items()}

    def norm(v, w):
        return v / (v * v).mean(1, keepdim=True).add(1e-6).sqrt() * w

    x = norm(leaf["residual"], leaf["norm_in"])
    w = torch.softmax((x @ leaf["router"].t()).gather(1, idx), 1)
    moe_rows = []
    for t in range(x.shape[0]):
        act = torch.nn.functional.silu(W["gate"][idx[t]] @ x[t]) * (W["up"][idx[t]] @ x[t])
        moe_rows.append((w[t, :, None] * (W["down"][idx[t]] @ act[:, :, None])[:, :, 0]).sum(0))
    added = norm(torch.stack(moe_rows), leaf["norm_out"])
    (leaf["residual"] + added).backward(c.d_out.double().cpu())
    rel = rel_l2(_np(out) - _np(c.residual), _np(added))
    print(f"training forward rel_l2={rel:.3e}", flush=True)
    assert rel <= 4 * Q
    # of the residual, what comes through the block
    past = _np(c.d_out)
    for name, t in leaf.items():
        got, ref = _np(grads[name]), _np(t.grad)
        if name == "residual":
            got, ref = got - past, ref - past
        rel = rel_l2(got, ref)
        print(f"gradient of {name} rel_l2={rel:.3e}", flush=True)
        assert rel <= 5 * Q, name
