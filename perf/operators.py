"""Speed cases of the MoE operators around the expert-LoRA fold: the router's
top-k choice (with its gradient), the sort of the routed rows by expert with
the dispatch of token rows, the weighted combine of expert rows (with its
gradient), and the products with 4-bit expert weights.

``own`` chooses the side: False computes the operators in their plain form,
elementary torch operations in 32 bits, rounded once at the end; True makes
the calls a user makes of moe_expert_lora_amd. ``exact`` is the definition in
64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
DEVICE = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _router(name, tokens, experts, top_k, dtype, renorm, backward):
    return dict(name=name, op="router", tokens=tokens, experts=experts, top_k=top_k, dtype=dtype,
                renorm=renorm, backward=backward)


def _dispatch(name, tokens, top_k, experts, dim, dtype, routing, dropped):
    return dict(name=name, op="dispatch", tokens=tokens, top_k=top_k, experts=experts, dim=dim,
                dtype=dtype, routing=routing, dropped=dropped)


def _combine(name, tokens, top_k, experts, dim, dtype, routing, dropped, by_slot, backward):
    return dict(name=name, op="combine", tokens=tokens, top_k=top_k, experts=experts, dim=dim,
                dtype=dtype, routing=routing, dropped=dropped, by_slot=by_slot,
                backward=backward)


def _w4(name, rows, experts, top_k, k_in, n_out, group, zeros, dtype, x_by_row):
    """experts == 0: one weight for every row (no indices)."""
    return dict(name=name, op="w4", rows=rows, experts=experts, top_k=top_k, k_in=k_in,
                n_out=n_out, group=group, zeros=zeros, dtype=dtype, x_by_row=x_by_row)


def listed():
    return [
        # the router of one decode step: 64 sequences padded to 80, top-8 of 128
        _router("router decode", 80, 128, 8, "bf16", True, False),
        # the router of a prefill batch of 8192 tokens
        _router("router prefill", 8192, 128, 8, "bf16", True, False),
        # the router's choice and its gradient in a training step, 256 experts
        _router("router train f32", 4096, 256, 8, "f32", False, True),
        # the rows of one decode step sorted by expert, for a step that groups them
        _dispatch("dispatch decode", 80, 8, 128, 768, "bf16", "uniform", 0.1),
        # a prefill batch of 4096 tokens, skewed routing: 32768 sorted rows
        _dispatch("dispatch prefill", 4096, 8, 128, 2048, "bf16", "zipf", 0.0),
        # the layer output of one decode step: rows in slot order
        _combine("combine decode", 80, 8, 128, 2048, "bf16", "uniform", 0.0, True, False),
        # the layer output of a prefill batch: rows in expert order
        _combine("combine prefill", 4096, 8, 128, 2048, "bf16", "zipf", 0.0, False, False),
        # the gradient of the weighted combine, 256 experts, some slots dropped
        _combine("combine train", 2048, 8, 256, 4096, "bf16", "uniform", 0.02, False, True),
        # one row through one 4-bit weight: a single sequence's projection
        _w4("w4 single row", 1, 0, 1, 2048, 2048, 128, False, "bf16", False),
        # ragged float32 rows, small groups with zero points, few experts
        _w4("w4 ragged f32", 37, 5, 1, 1000, 1365, 32, True, "f32", True),
        # the down projection of one decode step: 640 rows over 128 experts
        _w4("w4 decode down", 640, 128, 8, 768, 2048, 128, False, "bf16", True),
        # the gate/up projection of 256 sequences: 2048 rows over 128 experts
        _w4("w4 gate/up", 2048, 128, 8, 2048, 768, 64, True, "bf16", False),
    ]


def _log(rng, lo, hi):
    """lo .. hi, spread over the logarithm; never a multiple of 128, which the
    listed cases have."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v + 1 if v % 128 == 0 else v


def draw(rng):
    op = rng.choice(["router", "dispatch", "combine", "w4"])
    top = [work(c) for c in listed() if c["op"] == op]
    limit = {k: max(w[k] for w in top) for k in ("bytes", "flops")}
    while True:  # a draw beyond the largest listed case of its operator is drawn again
        c = _draw(rng, op)
        w = work(c)
        if w["bytes"] <= limit["bytes"] and (op != "w4" or w["flops"] <= limit["flops"]):
            return c


def _draw(rng, op):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "router":
        experts = _log(rng, 4, 511)
        top_k = min(experts, rng.choice([1, 2, 4, 6, 8]))
        # with top_k == 1 a renormalised weight is always 1, its gradient 0
        c = _router("", _log(rng, 1, 8190), experts, top_k, dtype,
                    top_k > 1 and rng.random() < 0.5, rng.random() < 0.5)
    elif op in ("dispatch", "combine"):
        experts = _log(rng, 4, 255)
        top_k = min(experts, rng.choice([1, 2, 4, 6, 8]))
        dim, tokens = _log(rng, 8, 511) * 8, _log(rng, 1, 16383)
        dropped = rng.choice([0.0, 0.0, 0.05, 0.3])
        routing = rng.choice(["uniform", "zipf"])
        if op == "dispatch":
            c = _dispatch("", tokens, top_k, experts, dim, dtype, routing, dropped)
        else:
            by_slot = rng.random() < 0.3
            c = _combine("", tokens, top_k, experts, dim, dtype, routing,
                         0.0 if by_slot else dropped, by_slot, rng.random() < 0.5)
    else:
        experts = rng.choice([0, 0, _log(rng, 2, 127)])
        top_k = 1 if experts == 0 else min(experts, rng.choice([1, 2, 4, 8]))
        rows = -(-_log(rng, 1, 2047 if experts else 63) // top_k) * top_k
        c = _w4("", rows, experts, top_k, _log(rng, 16, 511) * 8, _log(rng, 64, 4095),
                rng.choice([32, 64, 128, 256]), rng.random() < 0.5, dtype, rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 2654435761 % (2 ** 31) + 17)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE) * std).to(_TORCH[dtype])


def _choices(g, tokens, experts, top_k, routing, dropped):
    """Flat expert ids [tokens * top_k], int32: distinct per token; a dropped
    slot (a skipped sequence or a full expert) holds -1."""
    u = torch.rand((tokens, experts), generator=g, device=DEVICE).clamp_min_(1e-30)
    score = -torch.log(-torch.log(u))
    if routing == "zipf":
        score = score - 1.1 * torch.log(torch.arange(1, experts + 1, device=DEVICE).float())
    ids = torch.topk(score, top_k, dim=1).indices.to(torch.int32).reshape(-1)
    if dropped > 0:
        drop = torch.rand(ids.shape, generator=g, device=DEVICE) < dropped
        ids = torch.where(drop, torch.full_like(ids, -1), ids)
    return ids.contiguous()


def _sorted(ids, experts):
    """Offsets, sorted flat ids (-1 past the routed rows) and the row of each
    slot (-1 for a dropped slot)."""
    n = ids.numel()
    key = torch.where((ids >= 0) & (ids < experts), ids, torch.full_like(ids, experts)).long()
    order = torch.sort(key, stable=True).indices
    bounds = torch.arange(experts + 1, device=ids.device)
    offsets = (key.unsqueeze(0) < bounds.unsqueeze(1)).sum(1) if n * experts < 1 << 22 else \
        torch.cat([bounds[:1] * 0, torch.bincount(key, minlength=experts + 1)[:experts].cumsum(0)])
    pos = torch.arange(n, device=ids.device)
    sorted_ids = torch.where(pos < offsets[-1], order, torch.full_like(order, -1))
    rows = torch.empty_like(order)
    rows[order] = pos
    rows = torch.where(key < experts, rows, torch.full_like(rows, -1))
    return offsets.to(torch.int32), sorted_ids.to(torch.int32), rows.to(torch.int32)


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    d = {"case": case}
    if op == "router":
        # logits of a trained router: a few experts stand out per token
        d["logits"] = _normal(g, (case["tokens"], case["experts"]), case["dtype"], 2.0)
        if case["backward"]:
            d["d_weights"] = torch.randn((case["tokens"], case["top_k"]), generator=g,
                                         device=DEVICE)
    elif op == "dispatch":
        d["x"] = _normal(g, (case["tokens"], case["dim"]), case["dtype"])
        d["ids"] = _choices(g, case["tokens"], case["experts"], case["top_k"], case["routing"],
                            case["dropped"])
    elif op == "combine":
        slots = case["tokens"] * case["top_k"]
        ids = _choices(g, case["tokens"], case["experts"], case["top_k"], case["routing"],
                       case["dropped"])
        d["rows"] = _normal(g, (slots, case["dim"]), case["dtype"])
        d["weights"] = torch.softmax(
            torch.randn((case["tokens"], case["top_k"]), generator=g, device=DEVICE), 1)
        d["slot_rows"] = d["sorted_ids"] = None
        if not case["by_slot"]:
            _, d["sorted_ids"], d["slot_rows"] = _sorted(ids, case["experts"])
        if case["backward"]:
            d["d_out"] = _normal(g, (case["tokens"], case["dim"]), case["dtype"])
    else:
        k, n, e = case["k_in"], case["n_out"], max(1, case["experts"])
        groups = -(-k // case["group"])
        d["q"] = torch.randint(0, 256, (e, n, k // 2), generator=g, device=DEVICE,
                               dtype=torch.uint8)
        d["scales"] = ((torch.rand((e, n, groups), generator=g, device=DEVICE) + 0.5)
                       * (0.25 / math.sqrt(k))).to(_TORCH[case["dtype"]])
        d["zeros"] = torch.randint(0, 16, (e, n, groups), generator=g, device=DEVICE,
                                   dtype=torch.uint8) if case["zeros"] else None
        x_rows = case["rows"] if case["x_by_row"] else case["rows"] // case["top_k"]
        d["x"] = _normal(g, (x_rows, k), case["dtype"])
        d["ids"] = None
        if case["experts"]:
            tokens = case["rows"] // case["top_k"]
            d["ids"] = _choices(g, tokens, case["experts"], case["top_k"], "uniform", 0.02)
    return d


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The buffers and the weight layout a serving or training program keeps."""
    import moe_expert_lora_amd as ml
    c = s["case"]
    i32, f32 = torch.int32, torch.float32
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device=DEVICE)  # noqa: E731
    if c["op"] == "router":
        s["indices"] = new((c["tokens"], c["top_k"]), i32)
        s["weights"] = new((c["tokens"], c["top_k"]), f32)
        s["d_logits"] = torch.empty_like(s["logits"])
    elif c["op"] == "dispatch":
        n = s["ids"].numel()
        s["offsets"], s["sorted_ids"] = new((c["experts"] + 1,), i32), new((n,), i32)
        s["slot_rows"] = new((n,), i32)
        s["out_rows"] = new((n, c["dim"]), _TORCH[c["dtype"]])
        s["workspace"] = new((ml.mlora_moe_sort_workspace_bytes(n, c["experts"]),), torch.uint8)
    elif c["op"] == "combine":
        s["out"] = new((c["tokens"], c["dim"]), _TORCH[c["dtype"]])
        if c["backward"]:
            s["d_rows"] = torch.empty_like(s["rows"])
            s["d_weights"] = torch.empty_like(s["weights"])
    else:
        s["route"] = ml.make_w4_route(s.pop("q"), s.pop("scales"), s.pop("zeros"), c["k_in"],
                                      c["group"])
        s["out"] = new((c["rows"], c["n_out"]), _TORCH[c["dtype"]])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_router(s):
    import moe_expert_lora_amd as ml
    c = s["case"]
    ml.mlora_router_topk(s["logits"], s["indices"], s["weights"], renormalize=c["renorm"])
    if not c["backward"]:
        return s["indices"], s["weights"]
    ml.mlora_router_topk_backward(s["logits"], s["indices"], s["d_weights"], s["d_logits"],
                                  renormalize=c["renorm"])
    return s["indices"], s["weights"], s["d_logits"]


def _own_dispatch(s):
    import moe_expert_lora_amd as ml
    c = s["case"]
    ml.mlora_moe_sort(s["ids"], c["experts"], s["offsets"], s["sorted_ids"], s["slot_rows"],
                      s["workspace"])
    ml.mlora_moe_dispatch(s["x"], s["out_rows"], s["sorted_ids"], s["slot_rows"], c["top_k"])
    return s["offsets"], s["sorted_ids"], s["slot_rows"], s["out_rows"]


def _own_combine(s):
    import moe_expert_lora_amd as ml
    c = s["case"]
    if not c["backward"]:
        ml.mlora_moe_combine(s["rows"], s["out"], c["top_k"], s["weights"], s["slot_rows"])
        return s["out"]
    ml.mlora_moe_combine_backward(s["d_out"], s["rows"], s["weights"], s["d_rows"],
                                  s["d_weights"], c["top_k"], s["slot_rows"], s["sorted_ids"])
    return s["d_rows"], s["d_weights"]


def _own_w4(s):
    import moe_expert_lora_amd as ml
    c = s["case"]
    ml.mlora_w4_gather_gemv(s["route"], s["x"], s["out"], s["ids"], c["top_k"],
                            x_by_row=c["x_by_row"])
    return s["out"]


def _plain_router(s):
    c = s["case"]
    k = c["top_k"]
    lg = s["logits"].float()
    order = torch.sort(lg, dim=1, descending=True, stable=True).indices[:, :k]
    p = torch.softmax(lg, 1)
    w = torch.gather(p, 1, order)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    if not c["backward"]:
        return order.to(torch.int32), w
    dw = s["d_weights"]
    dot = (dw * w).sum(1, keepdim=True)
    if c["renorm"]:
        d = torch.zeros_like(lg).scatter_(1, order, w * (dw - dot))
    else:
        d = (torch.zeros_like(lg).scatter_(1, order, dw) - dot) * p
    return order.to(torch.int32), w, d.to(s["logits"].dtype)


def _plain_dispatch(s):
    c = s["case"]
    offsets, sorted_ids, slot_rows = _sorted(s["ids"], c["experts"])
    tok = torch.div(sorted_ids.clamp_min(0), c["top_k"], rounding_mode="floor").long()
    rows = torch.where(sorted_ids.unsqueeze(1) >= 0, s["x"][tok],
                       torch.zeros((), dtype=s["x"].dtype, device=DEVICE))
    return offsets, sorted_ids, slot_rows, rows


def _plain_combine(s):
    c = s["case"]
    t, k, dim = c["tokens"], c["top_k"], c["dim"]
    rows, w = s["rows"], s["weights"]
    if s["slot_rows"] is None:
        src, live = rows.view(t, k, dim).float(), None
    else:
        live = (s["slot_rows"] >= 0).view(t, k)
        src = rows[s["slot_rows"].clamp_min(0).long()].view(t, k, dim).float()
        src = torch.where(live.unsqueeze(2), src, torch.zeros((), device=DEVICE))
    if not c["backward"]:
        return (src * w.unsqueeze(2)).sum(1).to(rows.dtype)
    dout = s["d_out"].float().unsqueeze(1)
    dw = (src * dout).sum(2)
    per_slot = (dout * w.unsqueeze(2)).to(rows.dtype).view(t * k, dim)
    if live is None:
        return per_slot, dw
    ids = s["sorted_ids"]
    d_rows = torch.where(ids.unsqueeze(1) >= 0, per_slot[ids.clamp_min(0).long()],
                         torch.zeros((), dtype=rows.dtype, device=DEVICE))
    return d_rows, dw


def _plain_w4(s):
    c = s["case"]
    k, group = c["k_in"], c["group"]
    x = s["x"].float()
    q, sc, z = s["q"], s["scales"].float(), s["zeros"]

    def weights(e):
        """float32 weights of the experts e (a slice or ids): [.., n_out, k_in]"""
        b = q[e]
        v = torch.stack((b & 15, b >> 4), -1).flatten(-2).float()
        zero = 8.0 if z is None else z[e].float().repeat_interleave(group, -1)[..., :k]
        return (v - zero) * sc[e].repeat_interleave(group, -1)[..., :k]

    if s["ids"] is None:
        xr = x if c["x_by_row"] or c["top_k"] == 1 else x.repeat_interleave(c["top_k"], 0)
        return torch.matmul(xr, weights(0).t()).to(s["x"].dtype)
    xr = x if c["x_by_row"] else x.repeat_interleave(c["top_k"], 0)
    ids = s["ids"]
    step = max(1, (1 << 27) // (k * c["n_out"]))
    out = []
    for r in range(0, c["rows"], step):
        i = ids[r:r + step]
        w = weights(i.clamp_min(0).long())
        y = torch.matmul(w, xr[r:r + step].unsqueeze(2)).squeeze(2)
        out.append(torch.where(i.unsqueeze(1) >= 0, y, torch.zeros((), device=DEVICE)))
    return torch.cat(out).to(s["x"].dtype)


_OWN = {"router": _own_router, "dispatch": _own_dispatch, "combine": _own_combine, "w4": _own_w4}
_PLAIN = {"router": _plain_router, "dispatch": _plain_dispatch, "combine": _plain_combine,
          "w4": _plain_w4}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    es = _SIZE[case["dtype"]]
    if op == "router":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        b = t * e * es + t * k * 8
        f = 4 * t * e
        if case["backward"]:  # the logits again as gradient, the weights' gradient
            b += t * e * es + t * k * 4
            f += 4 * t * e
        return {"bytes": b, "flops": f}
    if op in ("dispatch", "combine"):
        t, k, dim = case["tokens"], case["top_k"], case["dim"]
        live = t * k * (1.0 - case["dropped"])
        if op == "dispatch":
            b = t * dim * es + t * k * dim * es + 3 * t * k * 4 + case["experts"] * 4
            return {"bytes": int(b), "flops": t * k}
        ids = 0 if case["by_slot"] else t * k * 4
        if not case["backward"]:
            return {"bytes": int(live * dim * es + t * dim * es + t * k * 4 + ids),
                    "flops": int(2 * live * dim)}
        return {"bytes": int(live * dim * es + t * k * dim * es + t * dim * es + t * k * 8 + 2 * ids),
                "flops": int(3 * live * dim)}
    k, n, rows = case["k_in"], case["n_out"], case["rows"]
    groups = -(-k // case["group"])
    e = 1.0
    if case["experts"]:  # experts that hold a row, on average
        miss = (1.0 - case["top_k"] / case["experts"]) ** (rows // case["top_k"])
        e = case["experts"] * (1.0 - miss)
    per = n * k / 2 + n * groups * (es + (1 if case["zeros"] else 0))
    x_rows = rows if case["x_by_row"] else rows // case["top_k"]
    return {"bytes": int(e * per + (x_rows * k + rows * n) * es + (rows * 4 if case["experts"] else 0)),
            "flops": 2 * rows * k * n}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    d = _inputs(case, seed)
    return {"router": _exact_router, "dispatch": _exact_dispatch, "combine": _exact_combine,
            "w4": _exact_w4}[case["op"]](case, d)


def _exact_router(c, d):
    lg = d["logits"].double().cpu().numpy()
    t, k = lg.shape[0], c["top_k"]
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :k]
    p = np.exp(lg - lg.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    at = np.arange(t)[:, None]
    w = p[at, idx]
    if c["renorm"]:
        w = w / w.sum(1, keepdims=True)
    if not c["backward"]:
        return None, torch.from_numpy(w)
    dw = d["d_weights"].double().cpu().numpy()
    # gradient of sum(dw * w) by the chain rule through the Jacobian of the choice
    jac = np.zeros_like(p)
    if c["renorm"]:
        total = p[at, idx].sum(1, keepdims=True)
        dp = dw / total - (dw * p[at, idx]).sum(1, keepdims=True) / total ** 2
    else:
        dp = dw
    jac[at, idx] = dp
    grad = p * jac - p * (p * jac).sum(1, keepdims=True)
    return None, torch.from_numpy(w), torch.from_numpy(grad)


def _exact_dispatch(c, d):
    ids = d["ids"].cpu().numpy()
    x = d["x"].double().cpu()
    live = [np.flatnonzero(ids == e) for e in range(c["experts"])]
    flat = np.concatenate(live)
    rows = torch.zeros((ids.size, c["dim"]), dtype=torch.float64)
    rows[: flat.size] = x[torch.from_numpy(flat // c["top_k"])]
    return None, None, None, rows


def _exact_combine(c, d):
    t, k = c["tokens"], c["top_k"]
    rows, w = d["rows"].double(), d["weights"].double()
    where = torch.arange(t * k, device=DEVICE) if d["slot_rows"] is None else d["slot_rows"].long()
    if not c["backward"]:
        out = torch.zeros((t, c["dim"]), dtype=torch.float64, device=DEVICE)
        for j in range(k):
            r = where[j::k]
            on = r >= 0
            out[on] += w[on, j, None] * rows[r[on]]
        return out
    g = d["d_out"].double()
    d_rows = torch.zeros_like(rows)
    dw = torch.zeros((t, k), dtype=torch.float64, device=DEVICE)
    for j in range(k):
        r = where[j::k]
        on = r >= 0
        d_rows[r[on]] = w[on, j, None] * g[on]
        dw[on, j] = (g[on] * rows[r[on]]).sum(1)
    return d_rows, dw


def _exact_w4(c, d):
    k, n = c["k_in"], c["n_out"]
    out = torch.zeros((c["rows"], n), dtype=torch.float64, device=DEVICE)
    row_x = torch.arange(c["rows"], device=DEVICE)
    if not c["x_by_row"]:
        row_x = torch.div(row_x, c["top_k"], rounding_mode="floor")
    group_of = torch.arange(k, device=DEVICE) // c["group"]
    for e in range(max(1, c["experts"])):
        r = torch.arange(c["rows"], device=DEVICE) if d["ids"] is None else \
            torch.nonzero(d["ids"] == e).flatten()
        if r.numel() == 0:
            continue
        w = torch.empty((n, k), dtype=torch.float64, device=DEVICE)
        w[:, 0::2] = (d["q"][e] % 16).double()
        w[:, 1::2] = torch.div(d["q"][e], 16, rounding_mode="floor").double()
        w -= 8.0 if d["zeros"] is None else d["zeros"][e].double()[:, group_of]
        w *= d["scales"][e].double()[:, group_of]
        out[r] = d["x"][row_x[r]].double() @ w.t()
    return out
