"""A MoE layer with expert LoRA, out of this library's calls.

``DecodeLayer`` runs one decode step: the router's choice, gate and up as 4-bit
products with their adapters folded in, the down projection with its own, and
the weighted combine. ``train_step`` routes a batch through any expert function
on rows sorted by expert and returns the gradients of the layer's output:
of the expert rows, the combine weights, the router's logits and the tokens.

``Fp8Block`` is a whole MoE block between residual rows, its experts' weights in
8 bits: ``prefill`` (norm, router, quantised rows, grouped products with their
adapters folded in, combine, norm and residual), ``decode`` of a few tokens, and
``train``, the gradients of a step whose expert weights stay frozen.

Run on an MI355X: ``python examples/moe_layer.py``.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_lora_amd as ml  # noqa: E402


class DecodeLayer:
    """One layer's packed weights, adapters and the buffers of a decode batch of
    up to ``max_tokens`` tokens.

    router: [n_experts, dim] bf16; gate, up, down: W4Route; lora: a dict of
    ExpertRoute for the same names (absent: no adapter there)."""

    def __init__(self, router, gate, up, down, lora, top_k, max_tokens):
        self.router, self.gate, self.up, self.down = router, gate, up, down
        self.lora, self.top_k = lora, top_k
        dev, bf16 = router.device, torch.bfloat16
        dim, hidden, slots = gate.k_in, gate.n_out, max_tokens * top_k
        self.indices = torch.empty((max_tokens, top_k), dtype=torch.int32, device=dev)
        self.weights = torch.empty((max_tokens, top_k), device=dev)
        self.gate_up = torch.empty((slots, 2 * hidden), dtype=bf16, device=dev)
        self.rows = torch.empty((slots, dim), dtype=bf16, device=dev)
        self.out = torch.empty((max_tokens, dim), dtype=bf16, device=dev)

    def _fold(self, names, x, outs, ids, row_adapter, x_by_row):
        calls = [ml.make_projection(self.lora[n], x, o, ids, row_adapter, self.top_k, x_by_row)
                 for n, o in zip(names, outs) if n in self.lora]
        if calls:
            ml.mlora_gather_bgmv_set(calls)

    def __call__(self, x, row_adapter):
        """x [tokens, dim] bf16, row_adapter [tokens] (0: the adapter, -1: none;
        mlora_build_moe_row_adapter_decode). Returns a view of a buffer."""
        t, k, hidden = x.shape[0], self.top_k, self.gate.n_out
        idx, w = self.indices[:t], self.weights[:t]
        ml.mlora_router_topk(x @ self.router.t(), idx, w, renormalize=True)
        ids = idx.view(-1)
        gate_up, rows, out = self.gate_up[:t * k], self.rows[:t * k], self.out[:t]
        gate, up = gate_up[:, :hidden], gate_up[:, hidden:]
        ml.mlora_w4_gather_gemv(self.gate, x, gate, ids, k)
        ml.mlora_w4_gather_gemv(self.up, x, up, ids, k)
        self._fold(("gate", "up"), x, (gate, up), ids, row_adapter, False)
        act = torch.nn.functional.silu(gate) * up
        ml.mlora_w4_gather_gemv(self.down, act, rows, ids, k, x_by_row=True)
        self._fold(("down",), act, (rows,), ids, row_adapter, True)
        ml.mlora_moe_combine(rows, out, k, w)
        return out


def train_step(x, logits, d_out, top_k, experts):
    """Routes x [tokens, dim] by logits [tokens, n_experts] through ``experts``
    and back, and the gradients for d_out [tokens, dim].

    experts(rows, offsets) -> (expert rows, backward), the rows sorted by expert
    (expert e's are offsets[e] .. offsets[e + 1]) and backward(d_rows) the
    gradient of its input rows. d_out may be a function that returns it for the
    layer's output. Returns (out, dict of gradients)."""
    t, dim = x.shape
    E, n, dev = logits.shape[1], x.shape[0] * top_k, x.device
    i32 = torch.int32
    idx, w = torch.empty((t, top_k), dtype=i32, device=dev), torch.empty((t, top_k), device=dev)
    ml.mlora_router_topk(logits, idx, w, renormalize=True)
    offsets = torch.empty(E + 1, dtype=i32, device=dev)
    sorted_ids, slots = torch.empty(n, dtype=i32, device=dev), torch.empty(n, dtype=i32, device=dev)
    ws = torch.empty(ml.mlora_moe_sort_workspace_bytes(n, E), dtype=torch.uint8, device=dev)
    ml.mlora_moe_sort(idx.view(-1), E, offsets, sorted_ids, slots, ws)
    rows = torch.empty((n, dim), dtype=x.dtype, device=dev)
    ml.mlora_moe_dispatch(x, rows, sorted_ids, slots, top_k)
    y, experts_backward = experts(rows, offsets)
    out = torch.empty_like(x)
    ml.mlora_moe_combine(y, out, top_k, w, slots)
    if callable(d_out):
        d_out = d_out(out)

    d_y, d_w = torch.empty_like(y), torch.empty_like(w)
    ml.mlora_moe_combine_backward(d_out, y, w, d_y, d_w, top_k, slots, sorted_ids)
    d_logits = torch.empty_like(logits)
    ml.mlora_router_topk_backward(logits, idx, d_w, d_logits, renormalize=True)
    d_x = torch.empty_like(x)
    ml.mlora_moe_combine(experts_backward(d_y), d_x, top_k, None, slots)  # dispatch's gradient
    return out, {"rows": d_y, "weights": d_w, "logits": d_logits, "x": d_x}


def fp8_product(route, rows, offsets=None, sorted_ids=None, top_k=1, up=None):
    """Products of an Fp8Route with ``rows`` (with ``up``: silu(rows) * up), which
    are quantised first; the outputs are sorted by expert as ``offsets`` says, row r
    of token sorted_ids[r] // top_k (None: of row r)."""
    n, k, dev = rows.shape[0], route.k_in, rows.device
    q = torch.empty((n, ml.mlora_fp8_row_width(k)), dtype=torch.float8_e4m3fn, device=dev)
    scales = torch.empty((-(-k // 128), n), device=dev)
    ml.mlora_fp8_quant(rows, q, scales, up=up)
    out = torch.empty((n if sorted_ids is None else sorted_ids.numel(), route.n_out),
                      dtype=rows.dtype, device=dev)
    ml.mlora_fp8_gemm(route, q, scales, out, offsets, sorted_ids, top_k)
    return out


def fp8_experts(gate, up, down, gate_t, up_t, down_t):
    """Frozen 8-bit experts for train_step: rows through gate, up, silu and down, and
    back through the transposed routes (make_fp8_route(..., transpose=True)). What a
    product reads is quantised, its gradient is taken as if it were not."""
    silu = torch.nn.functional.silu

    def experts(rows, offsets):
        g, u = fp8_product(gate, rows, offsets), fp8_product(up, rows, offsets)

        def backward(d_rows):
            d_act = fp8_product(down_t, d_rows, offsets)
            s = torch.sigmoid(g.float())
            d_g = (d_act * u * s * (1 + g * (1 - s))).to(rows.dtype)
            d_u = d_act * silu(g)
            return fp8_product(gate_t, d_g, offsets) + fp8_product(up_t, d_u, offsets)

        return fp8_product(down, g, offsets, up=u), backward

    return experts


class Fp8Block:
    """out = residual + norm(moe(norm(residual))), the experts' weights in 8 bits.

    norm_in, norm_out: [dim] norm weights; router: [n_experts, dim]; routes: dict of
    Fp8Route "gate", "up", "down" (and "gate_t", "up_t", "down_t" to train); lora: a
    dict of ExpertRoute (absent: no adapter there)."""

    MAX_DECODE = 16  # mlora_moe_layer's tokens

    def __init__(self, norm_in, norm_out, router, routes, lora, top_k):
        self.norm_in, self.norm_out, self.router = norm_in, norm_out, router
        self.routes, self.lora, self.top_k = routes, lora, top_k
        dim, hidden = routes["gate"].k_in, routes["gate"].n_out
        t, dev = self.MAX_DECODE, router.device
        self.x = torch.empty((t, dim), dtype=torch.bfloat16, device=dev)
        self.y, self.out = torch.empty_like(self.x), torch.empty_like(self.x)
        self.workspace = torch.empty(ml.mlora_moe_layer_workspace_bytes(
            t, router.shape[0], top_k, dim, hidden), dtype=torch.uint8, device=dev)

    def decode(self, residual):
        """Up to MAX_DECODE tokens without adapters, [tokens, dim] bf16. Returns a view
        of a buffer."""
        t = residual.shape[0]
        x, y, out = self.x[:t], self.y[:t], self.out[:t]
        ml.mlora_block_norm(residual, x=x, x_weight=self.norm_in)
        gate, up, down = (self.routes[n] for n in ("gate", "up", "down"))
        ml.mlora_moe_layer(gate, up, down, x, x @ self.router.t(), y, self.top_k, self.workspace,
                           renormalize=True)
        ml.mlora_block_norm(residual, r=out, y=y, y_weight=self.norm_out)
        return out

    def _fold(self, name, x, rows, offsets, ids, row_adapter, top_k):
        if name in self.lora:
            route, cap = self.lora[name], 8192
            ws = torch.empty(ml.mlora_grouped_down_all_workspace_bytes(
                rows.shape[0], cap, route.max_rank), dtype=torch.uint8, device=x.device)
            ml.mlora_grouped_down_all(route, x, rows, offsets, ids, row_adapter, top_k, cap, ws)

    def prefill(self, residual, row_adapter):
        """residual [tokens, dim] bf16, row_adapter [tokens] (0: the adapter, -1: none;
        mlora_build_moe_row_adapter_host)."""
        t, k, E, dev = residual.shape[0], self.top_k, self.router.shape[0], residual.device
        n, i32 = t * k, torch.int32
        x = torch.empty_like(residual)
        ml.mlora_block_norm(residual, x=x, x_weight=self.norm_in)
        idx, w = torch.empty((t, k), dtype=i32, device=dev), torch.empty((t, k), device=dev)
        ml.mlora_router_topk(x @ self.router.t(), idx, w, renormalize=True)
        offsets = torch.empty(E + 1, dtype=i32, device=dev)
        ids, slots = torch.empty(n, dtype=i32, device=dev), torch.empty(n, dtype=i32, device=dev)
        ws = torch.empty(ml.mlora_moe_sort_workspace_bytes(n, E), dtype=torch.uint8, device=dev)
        ml.mlora_moe_sort(idx.view(-1), E, offsets, ids, slots, ws)
        gate, up, down = (self.routes[m] for m in ("gate", "up", "down"))
        q = torch.empty((t, ml.mlora_fp8_row_width(gate.k_in)), dtype=torch.float8_e4m3fn,
                        device=dev)
        scales = torch.empty((-(-gate.k_in // 128), t), device=dev)
        ml.mlora_fp8_quant(x, q, scales)  # once for gate and up, and for a token's experts
        g = torch.empty((n, gate.n_out), dtype=x.dtype, device=dev)
        u = torch.empty_like(g)
        for name, route, rows in (("gate", gate, g), ("up", up, u)):
            ml.mlora_fp8_gemm(route, q, scales, rows, offsets, ids, k)
            self._fold(name, x, rows, offsets, ids, row_adapter, k)
        y = fp8_product(down, g, offsets, up=u)
        if "down" in self.lora:  # on the activated rows, which are sorted already
            self._fold("down", torch.nn.functional.silu(g) * u, y, offsets,
                       torch.arange(n, dtype=i32, device=dev),
                       row_adapter[(ids // k).long()], 1)
        moe = torch.empty_like(residual)
        ml.mlora_moe_combine(y, moe, k, w, slots)
        out = torch.empty_like(residual)
        ml.mlora_block_norm(residual, r=out, y=moe, y_weight=self.norm_out)
        return out

    def train(self, residual, d_out):
        """(out, gradients) for d_out: of the residual rows, both norms' weights and
        the router's."""
        x = torch.empty_like(residual)
        ml.mlora_block_norm(residual, x=x, x_weight=self.norm_in)
        ws = torch.empty(ml.mlora_block_norm_backward_workspace_bytes(*residual.shape),
                         dtype=torch.uint8, device=residual.device)
        out, d_residual = torch.empty_like(residual), torch.empty_like(residual)
        d_in, d_post = (torch.empty(residual.shape[1], device=residual.device) for _ in range(2))

        def d_moe(moe):
            ml.mlora_block_norm(residual, r=out, y=moe, y_weight=self.norm_out)
            d_y = torch.empty_like(moe)
            ml.mlora_block_norm_backward(residual, d_r=d_out, d_residual=d_residual, d_y=d_y,
                                         d_y_weight=d_post, y=moe, y_weight=self.norm_out,
                                         workspace=ws)
            return d_y

        experts = fp8_experts(*(self.routes[n] for n in ("gate", "up", "down", "gate_t", "up_t",
                                                         "down_t")))
        logits = x @ self.router.t()
        _, grads = train_step(x, logits, d_moe, self.top_k, experts)
        d_x = grads["x"] + grads["logits"] @ self.router
        # through the norm before the block, and past the block
        ml.mlora_block_norm_backward(residual, d_r=d_residual, d_x=d_x, d_residual=d_residual,
                                     d_x_weight=d_in, x_weight=self.norm_in, workspace=ws)
        return out, {"residual": d_residual, "norm_in": d_in, "norm_out": d_post,
                     "router": grads["logits"].t() @ x}


def adapter_route(a, b, scale=0.5):
    """ExpertRoute of adapters a [n_experts, rank, k] and b [n_experts, n, rank], and
    the tables that it points to."""
    import numpy as np
    E, rank, k = a.shape
    at, bt, st, cells = ml.mlora_pack_expert_tables(
        np.arange(E, dtype=np.int32), [a[e].data_ptr() for e in range(E)],
        [b[e].data_ptr() for e in range(E)], np.full(E, scale, np.float32))
    tables = [torch.from_numpy(v.view(np.int64)).to(a.device) for v in (at, bt)]
    tables.append(torch.from_numpy(st).to(a.device))
    return ml.make_route(*tables, cells, k, b.shape[1], rank, a.dtype), tables


def example_layer(n_experts=16, dim=512, hidden=256, rank=8, top_k=4, max_tokens=32, group=64,
                  seed=0):
    """A layer of random weights; returns it and the tensors it was made from."""
    dev, bf16 = "cuda", torch.bfloat16
    g = torch.Generator(device=dev).manual_seed(seed)
    made, packed, lora, keep = {}, {}, {}, []
    router = (torch.randn((n_experts, dim), generator=g, device=dev) * dim ** -0.5).to(bf16)
    for name, n, k in (("gate", hidden, dim), ("up", hidden, dim), ("down", dim, hidden)):
        q = torch.randint(0, 256, (n_experts, n, k // 2), generator=g, device=dev,
                          dtype=torch.uint8)
        scales = ((torch.rand((n_experts, n, -(-k // group)), generator=g, device=dev) + 0.5)
                  * 0.2 * k ** -0.5).to(bf16)
        a = (torch.randn((n_experts, rank, k), generator=g, device=dev) * k ** -0.5).to(bf16)
        b = (torch.randn((n_experts, n, rank), generator=g, device=dev) * 0.2).to(bf16)
        made[name] = (q, scales, a, b)
        packed[name] = ml.make_w4_route(q, scales, None, k, group)
        lora[name], tables = adapter_route(a, b)
        keep.append(tables)
    layer = DecodeLayer(router, packed["gate"], packed["up"], packed["down"], lora, top_k,
                        max_tokens)
    layer.keep = (made, keep)  # the device memory the routes point to
    return layer, router, made


def example_block(n_experts=16, dim=512, hidden=256, rank=8, top_k=4, seed=0):
    """An Fp8Block of random weights; returns it and the tensors it was made from."""
    dev, bf16 = "cuda", torch.bfloat16
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    router = (rnd(n_experts, dim) * dim ** -0.5).to(bf16)
    norms = [(1 + 0.2 * rnd(dim)).to(bf16) for _ in range(2)]
    made, routes, lora, keep = {}, {}, {}, []
    for name, n, k in (("gate", hidden, dim), ("up", hidden, dim), ("down", dim, hidden)):
        w = (rnd(n_experts, n, k) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        blocks = (n_experts, -(-n // 128), -(-k // 128))
        scales = (torch.rand(blocks, generator=g, device=dev) + 0.5) * 0.01 * k ** -0.5
        a, b = (rnd(n_experts, rank, k) * k ** -0.5).to(bf16), (rnd(n_experts, n, rank) * 0.2).to(bf16)
        made[name] = (w, scales, a, b)
        routes[name] = ml.make_fp8_route(w, scales)
        routes[name + "_t"] = ml.make_fp8_route(w, scales, transpose=True)
        lora[name], tables = adapter_route(a, b)
        keep.append(tables)
    block = Fp8Block(*norms, router, routes, lora, top_k)
    block.keep = (made, keep)  # the device memory the adapters' routes point to
    return block, made


def main():
    layer, router, _ = example_layer()
    x = torch.randn((24, router.shape[1]), device="cuda").to(torch.bfloat16)
    row_adapter = torch.from_numpy(
        ml.mlora_build_moe_row_adapter_decode([1] * 20 + [-1] * 4, 24, 1, True)).cuda()
    out = layer(x, row_adapter)
    print("decode step:", tuple(out.shape), "experts of token 0:", layer.indices[0].tolist())

    def experts(rows, offsets):  # any expert function; here one scale for all
        return rows * 2, lambda d_rows: d_rows * 2

    out, grads = train_step(x, x @ router.t(), torch.ones_like(x), 4, experts)
    print("training step:", tuple(out.shape), {k: tuple(v.shape) for k, v in grads.items()})

    block, _ = example_block()
    x = torch.randn((300, block.router.shape[1]), device="cuda").to(torch.bfloat16)
    row_adapter = torch.from_numpy(ml.mlora_build_moe_row_adapter_host([0, 200, 300], [0, -1])).cuda()
    print("8-bit block: prefill", tuple(block.prefill(x, row_adapter).shape), "decode",
          tuple(block.decode(x[:5]).shape))
    out, grads = block.train(x, torch.ones_like(x))
    print("8-bit block, training:", tuple(out.shape), {k: tuple(v.shape) for k, v in grads.items()})


if __name__ == "__main__":
    main()
