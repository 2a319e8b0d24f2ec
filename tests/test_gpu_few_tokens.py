"""GPU tests of the MoE layer for a few tokens, against its fp64 form and the
single calls."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8  # noqa: E402
from tests.fp8_cases import F32, U, close, to64, weights  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ml():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_lora_amd
    return moe_expert_lora_amd


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Case:
    def __init__(self, ml, seed, T, E, k, dim, hidden, dtype):
        rng = np.random.default_rng(seed)
        self.ml, self.k, self.dtype = ml, k, dtype
        made = {n: weights(rng, E, *s) for n, s in (("gate", (hidden, dim)), ("up", (hidden, dim)),
                                                    ("down", (dim, hidden)))}
        self.full = [fp8.expand(*made[n]) for n in ("gate", "up", "down")]
        self.routes = [ml.make_fp8_route(dev(w), dev(s)) for w, s in made.values()]
        self.x = dev(rng.normal(0, 1, (T, dim))).to(TORCH[dtype])
        self.logits = dev(rng.normal(0, 2, (T, E))).to(TORCH[dtype])
        self.out = torch.full((T, dim), 7.0, dtype=TORCH[dtype], device=DEV)
        self.idx = torch.full((T, k), -5, dtype=torch.int32, device=DEV)
        self.w = torch.full((T, k), -5.0, device=DEV)
        # whatever a workspace holds: bytes of a NaN
        self.ws = torch.full((ml.mlora_moe_layer_workspace_bytes(T, E, k, dim, hidden),), 0xff,
                             dtype=torch.uint8, device=DEV)

    def run(self, renorm=True, **kw):
        self.ml.mlora_moe_layer(*self.routes, self.x, self.logits, self.out, self.k, self.ws,
                                renormalize=renorm, indices=self.idx, weights=self.w, **kw)

    def check(self, renorm=True):
        self.run(renorm)
        ref, idx, w, mag = fp8.layer(to64(self.x), to64(self.logits), *self.full, self.k, renorm)
        assert np.array_equal(self.idx.cpu().numpy(), idx)
        close(to64(self.w), w, np.abs(w) * 64 * F32)
        # sums of dim and hidden products, the exponential's few roundings, and the
        # activated rows' parts: 2^-16 (fp32: 2^-24) of each value
        dim, hidden = self.x.shape[1], self.full[0].shape[1]
        parts = 2.0 ** -16 if self.dtype == "bf16" else F32
        err = mag * ((dim + hidden + 96) * F32 + parts)
        close(to64(self.out), ref, err + (np.abs(ref) + err) * U[self.dtype])


# tokens, experts, top_k, dim, hidden
CASES = [(1, 1, 1, 1, 1), (1, 8, 2, 256, 128), (3, 5, 5, 100, 40), (16, 16, 4, 300, 200),
         (7, 128, 8, 512, 96), (16, 129, 8, 128, 130), (2, 300, 17, 64, 48), (5, 1024, 6, 136, 24),
         (4, 70, 64, 40, 16), (16, 3, 2, 2100, 33), (9, 12, 3, 1000, 365), (1, 6, 1, 4096, 700),
         (13, 40, 40, 33, 65)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,dim,hidden", CASES)
def test_layer(ml, T, E, k, dim, hidden, dtype):
    c = Case(ml, T + E + dim, T, E, k, dim, hidden, dtype)
    c.check(True)
    c.check(False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", range(1, 17))
def test_every_number_of_tokens(ml, T, dtype):
    Case(ml, T, T, 10, 3, 144, 72, dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ties_masks_and_signed_zeros(ml, dtype):
    """Equal logits go to the lowest index; masked experts (-inf) come last with weight
    0; a token with nothing else has weights and a row of 0."""
    c = Case(ml, 1, 6, 9, 4, 72, 48, dtype)
    lg = c.logits
    lg[0] = 1.0
    lg[1] = -float("inf")
    lg[2, 3:] = -float("inf")
    lg[3, ::2], lg[3, 1::2] = 0.0, -0.0
    lg[4] = torch.finfo(lg.dtype).min
    c.check(True)
    c.check(False)
    assert c.idx[0].tolist() == [0, 1, 2, 3] and c.idx[1].tolist() == [0, 1, 2, 3]
    assert (c.w[1] == 0).all() and (c.out[1] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_are_not_finite_stay_alone(ml, dtype):
    c = Case(ml, 2, 8, 6, 2, 200, 150, dtype)
    c.run()
    want = c.out.clone()
    c.x[1, 7], c.x[4, 0], c.logits[6, 2] = float("nan"), float("inf"), float("nan")
    c.run()
    keep = [0, 2, 3, 5, 7]
    assert torch.equal(c.out[keep], want[keep])
    assert c.out[[1, 4, 6]].isnan().any(1).all()


def test_a_code_that_is_nan_reaches_only_its_expert(ml):
    rng = np.random.default_rng(3)
    E, dim, hidden, T = 4, 64, 32, 5
    made = [weights(rng, E, *s) for s in ((hidden, dim), (hidden, dim), (dim, hidden))]
    for w, _ in made:
        w[2] = 0x7f
    c = Case(ml, 3, T, E, 1, dim, hidden, "bf16")
    c.routes = [ml.make_fp8_route(dev(w), dev(s)) for w, s in made]
    c.logits.zero_()
    for t, e in enumerate((0, 2, 1, 3, 2)):
        c.logits[t, e] = 5
    c.run()
    bad = c.out.isnan()
    assert bad[[1, 4]].all() and not bad[[0, 2, 3]].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_what_lies_around(ml, dtype):
    """Rows of wider matrices that start off 16 bytes give the same bits; nothing
    outside the rows is written."""
    c = Case(ml, 4, 5, 20, 4, 264, 136, dtype)
    c.run()
    want = c.out.clone()
    for extra in (8, 3):
        wide = torch.full((7, 264 + 2 * extra), 5.0, dtype=c.x.dtype, device=DEV)
        out = wide[1:6, extra:extra + 264]
        x = torch.zeros_like(wide)[1:6, extra:extra + 264].copy_(c.x)
        lg = torch.zeros((5, 20 + extra), dtype=c.x.dtype, device=DEV)[:, extra:].copy_(c.logits)
        c.ml.mlora_moe_layer(*c.routes, x, lg, out, 4, c.ws, renormalize=True)
        assert torch.equal(out, want)
        out.fill_(5.0)
        assert (wide == 5).all()


def test_the_choice_is_the_routers(ml):
    for E, k in ((128, 8), (200, 20), (400, 3), (1000, 40)):
        c = Case(ml, E, 11, E, k, 24, 16, "bf16")
        for renorm in (False, True):
            c.run(renorm)
            idx, w = torch.empty_like(c.idx), torch.empty_like(c.w)
            ml.mlora_router_topk(c.logits, idx, w, renormalize=renorm)
            assert torch.equal(idx, c.idx) and torch.equal(w, c.w)


def test_streams_graphs_and_reruns(ml):
    """Replays of a captured graph with inputs changed in place, eager calls between
    them on the same workspace, and a side stream give the eager bits."""
    c = Case(ml, 5, 6, 30, 4, 256, 160, "bf16")
    c.run()
    want = c.out.clone()
    side = torch.cuda.Stream()
    c.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(c.out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for i in range(4):
        c.x.copy_(torch.randn_like(c.x))
        c.logits.copy_(torch.randn_like(c.logits))
        graph.replay()
        torch.cuda.synchronize()
        got = c.out.clone(), c.idx.clone(), c.w.clone()
        c.run()
        assert all(torch.equal(a, b) for a, b in zip(got, (c.out, c.idx, c.w))), i


def test_python_refuses(ml):
    c = Case(ml, 6, 4, 8, 2, 64, 32, "bf16")
    g, u, d = c.routes
    call = lambda **k: ml.mlora_moe_layer(*k.pop("routes", c.routes), k.pop("x", c.x),  # noqa: E731
                                          k.pop("logits", c.logits), k.pop("out", c.out),
                                          k.pop("top_k", 2), k.pop("ws", c.ws), **k)
    for error, kw in [(TypeError, dict(x=c.x.float())), (TypeError, dict(logits=c.logits.float())),
                      (ValueError, dict(out=c.out[:3])), (ValueError, dict(logits=c.logits[:, :7])),
                      (ValueError, dict(x=c.x[:, :63])), (ValueError, dict(indices=c.idx[:3])),
                      (TypeError, dict(weights=c.w.double())), (ValueError, dict(ws=c.ws.cpu())),
                      (ml.MloraError, dict(ws=None)), (ml.MloraError, dict(ws=c.ws[:-256])),
                      (ml.MloraError, dict(top_k=9)), (ml.MloraError, dict(routes=(g, u, g)))]:
        with pytest.raises(error):
            call(**kw)
    big = torch.zeros((17, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ml.MloraError):
        call(x=big, out=big.clone(), logits=torch.zeros((17, 8), dtype=torch.bfloat16, device=DEV))
