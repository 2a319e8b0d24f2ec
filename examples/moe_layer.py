"""A MoE layer with expert LoRA, out of this library's calls.

``DecodeLayer`` runs one decode step: the router's choice, gate and up as 4-bit
products with their adapters folded in, the down projection with its own, and
the weighted combine. ``train_step`` routes a batch through any expert function
on rows sorted by expert and returns the gradients of the layer's output:
of the expert rows, the combine weights, the router's logits and the tokens.

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
    gradient of its input rows. Returns (out, dict of gradients)."""
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

    d_y, d_w = torch.empty_like(y), torch.empty_like(w)
    ml.mlora_moe_combine_backward(d_out, y, w, d_y, d_w, top_k, slots, sorted_ids)
    d_logits = torch.empty_like(logits)
    ml.mlora_router_topk_backward(logits, idx, d_w, d_logits, renormalize=True)
    d_x = torch.empty_like(x)
    ml.mlora_moe_combine(experts_backward(d_y), d_x, top_k, None, slots)  # dispatch's gradient
    return out, {"rows": d_y, "weights": d_w, "logits": d_logits, "x": d_x}


def example_layer(n_experts=16, dim=512, hidden=256, rank=8, top_k=4, max_tokens=32, group=64,
                  seed=0):
    """A layer of random weights; returns it and the tensors it was made from."""
    import numpy as np
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
        at, bt, st, cells = ml.mlora_pack_expert_tables(
            np.arange(n_experts, dtype=np.int32), [a[e].data_ptr() for e in range(n_experts)],
            [b[e].data_ptr() for e in range(n_experts)], np.full(n_experts, 0.5, np.float32))
        tables = [torch.from_numpy(v.view(np.int64)).to(dev) for v in (at, bt)]
        tables.append(torch.from_numpy(st).to(dev))
        lora[name] = ml.make_route(*tables, cells, k, n, rank, bf16)
        keep.append(tables)
    layer = DecodeLayer(router, packed["gate"], packed["up"], packed["down"], lora, top_k,
                        max_tokens)
    layer.keep = (made, keep)  # the device memory the routes point to
    return layer, router, made


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


if __name__ == "__main__":
    main()
