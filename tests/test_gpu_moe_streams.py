"""GPU tests of the MoE layer's operators on a stream given by argument."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def ml():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_lora_amd
    return moe_expert_lora_amd


def _inputs(dtype, tokens, E, k, dim, n):
    g = torch.Generator(device=DEV).manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    byte = lambda *s: torch.randint(0, 256, s, generator=g, device=DEV,  # noqa: E731
                                    dtype=torch.uint8)
    return dict(logits=rnd(tokens, E).to(dtype), x=rnd(tokens, dim).to(dtype),
                d_out=rnd(tokens, n).to(dtype), q=byte(E, n, dim // 2),
                scales=(rnd(E, n, dim // 64).abs() * 0.02).to(dtype),
                zeros=byte(E, n, dim // 64) % 16)


def _step(ml, d, k, stream):
    """Every call once, each with ``stream``: packed on it, too."""
    dtype, tokens, E = d["logits"].dtype, d["x"].shape[0], d["logits"].shape[1]
    slots, n, dim = tokens * k, d["d_out"].shape[1], d["x"].shape[1]
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    new = lambda *s: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    o = dict(idx=i32(tokens, k), w=torch.zeros((tokens, k), device=DEV), off=i32(E + 1),
             order=i32(slots), rows=i32(slots), sent=new(slots, dim), y=new(slots, n),
             out=new(tokens, n), d_y=new(slots, n), d_w=torch.zeros((tokens, k), device=DEV),
             d_l=torch.zeros_like(d["logits"]))
    ws = torch.empty(ml.mlora_moe_sort_workspace_bytes(slots, E), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    route = ml.make_w4_route(d["q"], d["scales"], d["zeros"], dim, 64, stream=stream)
    ml.mlora_router_topk(d["logits"], o["idx"], o["w"], renormalize=True, stream=stream)
    ids = o["idx"].view(-1)
    ml.mlora_moe_sort(ids, E, o["off"], o["order"], o["rows"], ws, stream=stream)
    ml.mlora_moe_dispatch(d["x"], o["sent"], o["order"], o["rows"], k, stream=stream)
    ml.mlora_w4_gather_gemv(route, d["x"], o["y"], ids, k, stream=stream)
    ml.mlora_moe_combine(o["y"], o["out"], k, o["w"], stream=stream)
    ml.mlora_moe_combine_backward(d["d_out"], o["y"], o["w"], o["d_y"], o["d_w"], k, stream=stream)
    ml.mlora_router_topk_backward(d["logits"], o["idx"], o["d_w"], o["d_l"], renormalize=True,
                                  stream=stream)
    torch.cuda.synchronize()
    return o


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens", [5, 700])
def test_every_call_on_a_given_stream(ml, dtype, tokens):
    """On a side stream each call gives the current stream's bits."""
    d = _inputs(dtype, tokens, 16, 4, 256, 200)
    want = _step(ml, d, 4, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _step(ml, d, 4, side)
    for name, t in want.items():
        assert torch.equal(got[name], t), name


def test_packed_memory_belongs_to_the_given_stream(ml):
    """A dropped route's block goes back to the stream that wrote it, not to the
    current one, where a new tensor could be written while that stream reads."""
    E, n, k = 8, 2048, 4096                       # 33 MB: a block of its own
    q = torch.zeros((E, n, k // 2), dtype=torch.uint8, device=DEV)
    s = torch.ones((E, n, k // 128), dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    route = ml.make_w4_route(q, s, None, k, 128, stream=side)
    at, size = route._keep.data_ptr(), route._keep.numel()
    torch.cuda.synchronize()
    del route
    here = torch.empty(size, dtype=torch.uint8, device=DEV)
    assert here.data_ptr() != at
    with torch.cuda.stream(side):
        there = torch.empty(size, dtype=torch.uint8, device=DEV)
    assert there.data_ptr() == at
    torch.cuda.synchronize()
