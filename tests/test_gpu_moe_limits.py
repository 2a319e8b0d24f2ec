"""GPU tests of the MoE layer's operators at sizes whose threads do not fit one
grid dimension (2^32): tokens of the router and of the row movers, words of packed
4-bit weights. Checked on the device, against torch."""
from __future__ import annotations

import gc

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ml():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_lora_amd
    return moe_expert_lora_amd


@pytest.fixture(autouse=True)
def _room():
    """50 GB free before a test, and given back after it."""
    gc.collect()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 50e9:
        pytest.skip("needs 50 GB of device memory")
    yield
    gc.collect()
    torch.cuda.empty_cache()


def test_router_tokens(ml):
    """16 lanes a token: more than 2^28 tokens. Two experts, one chosen: the
    larger, with p = 1 / (1 + exp(-|difference|)); its gradient is +- dw p (1 - p).
    A quotient and an exponential of a difference below 16: 32 u; the gradient, of
    1 - p by cancellation, 64 u of dw, and half a bf16 step of itself."""
    tokens = (1 << 28) + 70
    g = torch.Generator(device=DEV).manual_seed(1)
    lg = torch.empty((tokens, 2), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    idx = torch.full((tokens, 1), -7, dtype=torch.int32, device=DEV)
    w = torch.full((tokens, 1), 9.0, device=DEV)
    ml.mlora_router_topk(lg, idx, w)
    dw = torch.empty((tokens, 1), device=DEV).normal_(generator=g)
    dl = torch.full_like(lg, 9.0)
    ml.mlora_router_topk_backward(lg, idx, dw, dl)
    step = 1 << 26
    for t in range(0, tokens, step):
        s = slice(t, t + step)
        second = lg[s, 1] > lg[s, 0]
        assert torch.equal(idx[s, 0] == 1, second) and int(idx[s].min()) >= 0
        p = torch.sigmoid((lg[s, 1].double() - lg[s, 0].double()).abs())
        assert float((w[s, 0] - p).abs().max()) <= 32 * U
        grad = dw[s, 0].double() * p * (1 - p) * torch.where(second, 1.0, -1.0)
        for e, ref in ((0, -grad), (1, grad)):
            tol = 64 * U * dw[s, 0].abs() + 2.0 ** -8 * ref.abs() + 2.0 ** -126
            assert bool(((dl[s, e].double() - ref).abs() <= tol).all())


def test_row_movers_tokens(ml):
    """256 threads a token: more than 2^24 tokens of more than 128 columns."""
    tokens, dim = (1 << 24) + 5, 129
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.empty((tokens, dim), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    ids = torch.randint(-1, 3, (tokens,), generator=g, device=DEV, dtype=torch.int32)
    off, order, slots = (torch.empty(n, dtype=torch.int32, device=DEV)
                         for n in (4, tokens, tokens))
    ws = torch.empty(ml.mlora_moe_sort_workspace_bytes(tokens, 3), dtype=torch.uint8, device=DEV)
    ml.mlora_moe_sort(ids, 3, off, order, slots, ws)
    live = ids >= 0
    n_live = int(live.sum())
    assert int(off[3]) == n_live and bool(((slots >= 0) == live).all())
    rows = torch.full((tokens, dim), 9.0, dtype=x.dtype, device=DEV)
    ml.mlora_moe_dispatch(x, rows, order, slots, 1)
    assert torch.equal(rows[:n_live], x[order[:n_live].long()])
    assert not bool(rows[n_live:].any())
    out = torch.full_like(x, 9.0)
    ml.mlora_moe_combine(rows, out, 1, None, slots)
    x[~live] = 0
    assert torch.equal(out, x)
    out.fill_(9.0)
    w = torch.full((tokens, 1), 0.5, device=DEV)
    d_w = torch.full((tokens, 1), 9.0, device=DEV)
    ml.mlora_moe_combine_backward(x, rows, w, out, d_w, 1, slots, order)
    assert torch.equal(out[:n_live], rows[:n_live] / 2) and not bool(out[n_live:].any())
    # 129 products of fp32 and their sums: 150 u of the (positive) sum
    for t in range(0, tokens, 1 << 22):
        want = (x[t:t + (1 << 22)].double() ** 2).sum(1)
        assert bool(((d_w[t:t + (1 << 22), 0] - want).abs() <= 150 * U * want).all())


def test_packed_words(ml):
    """More than 2^32 words of packed weights (17 GB): products of the first and the
    last experts. A bf16 output is off by half a step of itself, and by fp32 sums of
    8192 products: the probabilistic bound 10 sqrt(8192) u of their absolute sum."""
    E, n, k = 1024, 4100, 8192
    assert E * ((n + 31) // 32) * (k // 32) * 128 > 1 << 32
    g = torch.Generator(device=DEV).manual_seed(3)
    q = torch.empty((E, n, k // 2), dtype=torch.uint8, device=DEV)
    for e in range(0, E, 64):
        q[e:e + 64].random_(0, 256, generator=g)
    s = (torch.rand((E, n, 1), generator=g, device=DEV) * 0.01 + 0.01).to(torch.bfloat16)
    route = ml.make_w4_route(q, s, None, k, k)
    ids = torch.tensor([0, 1023, 5, 1022], dtype=torch.int32, device=DEV)
    x = torch.randn((4, k), generator=g, device=DEV).to(torch.bfloat16)
    out = torch.full((4, n), 9e9, dtype=torch.bfloat16, device=DEV)
    ml.mlora_w4_gather_gemv(route, x, out, ids)
    for r, e in enumerate(ids.tolist()):
        v = torch.stack((q[e] & 15, q[e] >> 4), -1).flatten(-2).double() - 8
        w = v * s[e].double()
        ref, mag = w @ x[r].double(), w.abs() @ x[r].double().abs()
        tol = 10 * 8192 ** 0.5 * U * mag
        assert bool(((out[r].double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol)).all())


def test_rows_wider_than_32_bits(ml):
    """2^32 + 8 experts are refused, not taken as 8."""
    wide = torch.empty((1, (1 << 32) + 8), dtype=torch.bfloat16, device=DEV)
    idx = torch.full((1, 4), -7, dtype=torch.int32, device=DEV)
    w = torch.full((1, 4), 9.0, device=DEV)
    with pytest.raises(ValueError, match="logits is too wide"):
        ml.mlora_router_topk(wide, idx, w)
    with pytest.raises(ValueError, match="logits is too wide"):
        ml.mlora_router_topk_backward(wide, idx, w, wide)
    torch.cuda.synchronize()
    assert bool((idx == -7).all()) and bool((w == 9).all())


def test_more_choices_than_32_bits(ml):
    """2^32 + 4 choices are refused, not taken as 4."""
    lg = torch.zeros((1, 16), device=DEV)
    idx = torch.empty((1, (1 << 32) + 4), dtype=torch.int32, device=DEV)
    w = torch.empty((1, (1 << 32) + 4), device=DEV)
    with pytest.raises(ValueError, match="indices is too wide"):
        ml.mlora_router_topk(lg, idx, w)
