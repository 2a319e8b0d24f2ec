"""Speed cases of the operators beside the MoE layer's: products with 8-bit
floating-point weights that have a scale for each block of 128 x 128 (the rows
quantised on the way in), a whole MoE layer for a few tokens, and the norms
after and before a block with its gate and residual scale (with gradients).

``own`` chooses the side: False computes the operators in their plain form,
elementary torch operations in 32 bits (64 where a value is next to a rounding
border), rounded once at the end; True makes the calls a user makes of
moe_expert_lora_amd. ``exact`` is the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
DEVICE = "cuda"
BLOCK = 128
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _product(name, rows, experts, top_k, k_in, n_out, source, dtype, routing="uniform",
             transposed=False):
    """experts == 0: one weight for every row. source: what the rows are
    quantised from: "tokens" (token rows, gathered by the product through the
    sorted ids), "rows" (as they lie) or "silu" (silu(gate) * up of each row).
    transposed: the gradient of the rows, through the same weights."""
    return dict(name=name, op="product", rows=rows, experts=experts, top_k=top_k, k_in=k_in,
                n_out=n_out, source=source, dtype=dtype, routing=routing, transposed=transposed)


def _layer(name, tokens, experts, top_k, dim, hidden, dtype, renorm):
    return dict(name=name, op="layer", tokens=tokens, experts=experts, top_k=top_k, dim=dim,
                hidden=hidden, dtype=dtype, renorm=renorm)


def _norm(name, tokens, dim, dtype, post, gate, backward):
    """post: the block's output is normed before it is added. gate: "none",
    "channel" [dim], "token" [tokens, 1] or "full" [tokens, dim]."""
    return dict(name=name, op="norm", tokens=tokens, dim=dim, dtype=dtype, post=post, gate=gate,
                backward=backward)


def listed():
    return [
        # one sequence's projection through one weight
        _product("fp8 single row", 1, 0, 1, 2048, 2048, "rows", "bf16"),
        # the down projection of one decode step: 640 activated rows over 128 experts
        _product("fp8 decode down", 640, 128, 8, 768, 2048, "silu", "bf16"),
        # the gate projection of a prefill batch of 4096 tokens, skewed routing
        _product("fp8 prefill gate", 32768, 128, 8, 2048, 768, "tokens", "bf16", "zipf"),
        # one weight for every token of a batch (a shared expert's): bound by the product
        _product("fp8 one weight", 8192, 0, 1, 4096, 4096, "rows", "bf16"),
        # the gradient of ragged float32 rows through a few experts
        _product("fp8 gradient f32", 2001, 5, 1, 1365, 1000, "rows", "f32", "uniform", True),
        # the MoE layer of a single sequence's decode step
        _layer("layer one token", 1, 128, 8, 2048, 768, "bf16", True),
        # of sixteen sequences
        _layer("layer 16 tokens", 16, 128, 8, 2048, 768, "bf16", True),
        # ragged float32, few experts
        _layer("layer ragged f32", 5, 12, 3, 1000, 365, "f32", False),
        # residual and the next norm in one decode step
        _norm("norm decode", 80, 2048, "bf16", False, "none", False),
        # norms on both sides and a gate per token, a prefill batch
        _norm("norm prefill", 8192, 4096, "bf16", True, "token", False),
        # the gradients of both norms and of a gate per channel in a training step
        _norm("norm train", 4096, 2048, "bf16", True, "channel", True),
        # ragged float32 with a full gate
        _norm("norm train f32", 777, 1365, "f32", True, "full", True),
    ]


def _log(rng, lo, hi):
    """lo .. hi, spread over the logarithm; never a multiple of 128, which the
    listed cases have."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v + 1 if v % 128 == 0 else v


def draw(rng):
    op = rng.choice(["product", "layer", "norm"])
    top = [work(c) for c in listed() if c["op"] == op]
    limit = {k: max(w[k] for w in top) for k in ("bytes", "flops")}
    while True:  # a draw beyond the largest listed case of its operator is drawn again
        c = _draw(rng, op)
        w = work(c)
        if w["bytes"] <= limit["bytes"] and w["flops"] <= limit["flops"]:
            return c


def _draw(rng, op):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "product":
        experts = rng.choice([0, _log(rng, 2, 127), _log(rng, 2, 127)])
        top_k = min(max(1, experts), rng.choice([1, 2, 4, 8])) if experts else 1
        source = rng.choice(["tokens", "rows", "silu"]) if experts else rng.choice(["rows", "silu"])
        if source == "silu":
            dtype = "bf16"  # what a gate / up product writes
        rows = -(-_log(rng, 1, 16383) // top_k) * top_k
        c = _product("", rows, experts, top_k, _log(rng, 40, 4095), _log(rng, 40, 4095), source,
                     dtype, rng.choice(["uniform", "zipf"]), source == "rows" and rng.random() < 0.5)
    elif op == "layer":
        experts = _log(rng, 4, 255)
        c = _layer("", rng.randint(1, 16), experts, min(experts, rng.choice([1, 2, 4, 6, 8])),
                   _log(rng, 100, 4095), _log(rng, 40, 2047), dtype, rng.random() < 0.5)
    else:
        c = _norm("", _log(rng, 1, 8190), _log(rng, 8, 8191), dtype, rng.random() < 0.5,
                  rng.choice(["none", "channel", "token", "full"]), rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 2654435761 % (2 ** 31) + 29)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE) * std).to(_TORCH[dtype])


def _weights(g, experts, n, k):
    """E4M3 codes as a block's quantiser leaves them (largest values near 448)
    and the blocks' scales, which make a row's norm about 1."""
    w = torch.empty((experts, n, k), dtype=torch.float8_e4m3fn, device=DEVICE)
    step = max(1, (1 << 26) // (n * k))
    for e in range(0, experts, step):
        part = w[e:e + step]
        part.copy_(torch.randn(part.shape, generator=g, device=DEVICE).mul_(110.).clamp_(-448, 448))
    s = torch.rand((experts, -(-n // BLOCK), -(-k // BLOCK)), generator=g, device=DEVICE) + 0.5
    return w, s / (110.0 * math.sqrt(k))


def _spans(g, case):
    """Offsets of the experts in the sorted rows, the sorted flat ids, and the
    offsets on the host: distinct experts per token."""
    experts, k = case["experts"], case["top_k"]
    tokens = case["rows"] // k
    u = torch.rand((tokens, experts), generator=g, device=DEVICE).clamp_min_(1e-30)
    score = -torch.log(-torch.log(u))
    if case["routing"] == "zipf":
        score = score - 1.1 * torch.log(torch.arange(1, experts + 1, device=DEVICE).float())
    ids = torch.topk(score, k, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=DEVICE)
    offsets[1:] = torch.bincount(ids, minlength=experts).cumsum(0)
    return offsets.to(torch.int32), order.to(torch.int32), offsets.tolist()


def _inputs(case, seed):
    g = _gen(seed)
    d = {"case": case}
    if case["op"] == "product":
        e, rows, k, n = max(1, case["experts"]), case["rows"], case["k_in"], case["n_out"]
        # transposed: the stored weight is the forward's, [k_in, n_out] here
        d["w"], d["w_scales"] = _weights(g, e, k, n) if case["transposed"] else _weights(g, e, n, k)
        d["offsets"], d["sorted_ids"], d["spans"] = None, None, [0, rows]
        if case["experts"]:
            d["offsets"], d["sorted_ids"], d["spans"] = _spans(g, case)
        if case["source"] == "tokens":
            d["x"] = _normal(g, (rows // case["top_k"], k), case["dtype"])
        else:
            d["x"] = _normal(g, (rows, k), case["dtype"])
        if case["source"] == "silu":
            d["up"] = _normal(g, (rows, k), case["dtype"])
    elif case["op"] == "layer":
        e, dim, h = case["experts"], case["dim"], case["hidden"]
        d["gate"], d["up"], d["down"] = _weights(g, e, h, dim), _weights(g, e, h, dim), \
            _weights(g, e, dim, h)
        d["x"] = _normal(g, (case["tokens"], dim), case["dtype"])
        # logits of a trained router: a few experts stand out per token
        d["logits"] = _normal(g, (case["tokens"], e), case["dtype"], 2.0)
    else:
        t, dim, dt = case["tokens"], case["dim"], case["dtype"]
        d["residual"], d["y"] = _normal(g, (t, dim), dt, 2.0), _normal(g, (t, dim), dt)
        d["x_weight"] = 1 + 0.1 * torch.randn(dim, generator=g, device=DEVICE)
        d["y_weight"] = 1 + 0.1 * torch.randn(dim, generator=g, device=DEVICE) \
            if case["post"] else None
        shape = {"none": None, "channel": (dim,), "token": (t, 1), "full": (t, dim)}[case["gate"]]
        d["gate"] = None if shape is None else _normal(g, shape, dt, 0.5)
        d["residual_scale"], d["y_scale"] = 0.75, 1.25
        if case["backward"]:
            d["d_r"], d["d_x"] = _normal(g, (t, dim), dt), _normal(g, (t, dim), dt)
    return d


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The weight layouts and buffers a serving or training program keeps."""
    import moe_expert_lora_amd as ml
    c = s["case"]
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device=DEVICE)  # noqa: E731
    if c["op"] == "product":
        s["route"] = ml.make_fp8_route(s.pop("w"), s.pop("w_scales"), transpose=c["transposed"])
        q_rows = s["x"].shape[0]
        s["q"] = new((q_rows, ml.mlora_fp8_row_width(c["k_in"])), torch.float8_e4m3fn)
        s["q_scales"] = new((-(-c["k_in"] // BLOCK), q_rows), torch.float32)
        s["out"] = new((c["rows"], c["n_out"]), _TORCH[c["dtype"]])
        if c["source"] != "tokens":
            s["sorted_ids"] = None
    elif c["op"] == "layer":
        for name in ("gate", "up", "down"):
            s[name] = ml.make_fp8_route(*s[name])
        t, k = c["tokens"], c["top_k"]
        s["out"] = torch.empty_like(s["x"])
        s["indices"], s["weights"] = new((t, k), torch.int32), new((t, k), torch.float32)
        s["workspace"] = new((ml.mlora_moe_layer_workspace_bytes(
            t, c["experts"], k, c["dim"], c["hidden"]),), torch.uint8)
    else:
        if c["backward"]:
            s["d_residual"], s["d_y"] = torch.empty_like(s["residual"]), torch.empty_like(s["y"])
            s["d_x_weight"] = torch.empty_like(s["x_weight"])
            s["d_y_weight"] = torch.empty_like(s["y_weight"]) if c["post"] else None
            s["d_gate"] = None if s["gate"] is None else torch.empty(
                s["gate"].shape, dtype=_TORCH[c["dtype"]] if c["gate"] == "full" else torch.float32,
                device=DEVICE)
            s["workspace"] = new((ml.mlora_block_norm_backward_workspace_bytes(
                c["tokens"], c["dim"]),), torch.uint8)
        else:
            s["r"], s["x"] = torch.empty_like(s["residual"]), torch.empty_like(s["residual"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_product(s):
    import moe_expert_lora_amd as ml
    c = s["case"]
    ml.mlora_fp8_quant(s["x"], s["q"], s["q_scales"], up=s.get("up"))
    ml.mlora_fp8_gemm(s["route"], s["q"], s["q_scales"], s["out"], s["offsets"], s["sorted_ids"],
                      c["top_k"])
    return s["out"]


def _own_layer(s):
    import moe_expert_lora_amd as ml
    c = s["case"]
    ml.mlora_moe_layer(s["gate"], s["up"], s["down"], s["x"], s["logits"], s["out"], c["top_k"],
                       s["workspace"], renormalize=c["renorm"], indices=s["indices"],
                       weights=s["weights"])
    return s["out"], s["indices"], s["weights"]


def _own_norm(s):
    import moe_expert_lora_amd as ml
    kw = dict(y=s["y"], x_weight=s["x_weight"], y_weight=s["y_weight"], gate=s["gate"],
              residual_scale=s["residual_scale"], y_scale=s["y_scale"], eps=EPS)
    if not s["case"]["backward"]:
        ml.mlora_block_norm(s["residual"], r=s["r"], x=s["x"], **kw)
        return s["r"], s["x"]
    ml.mlora_block_norm_backward(
        s["residual"], d_r=s["d_r"], d_x=s["d_x"], d_residual=s["d_residual"], d_y=s["d_y"],
        d_x_weight=s["d_x_weight"], d_y_weight=s["d_y_weight"], d_gate=s["d_gate"],
        workspace=s["workspace"], **kw)
    return s["d_residual"], s["d_y"], s["d_x_weight"], s["d_y_weight"], s["d_gate"]


def _plain_quant(x):
    """The E4M3 values of each group of 128 of the rows (float32) times their
    scale: 448 / (largest magnitude) x, rounded to even. The quotient is taken in
    64 bits, where no value crosses the border between two codes."""
    rows, k = x.shape
    pad = torch.zeros((rows, -k % BLOCK), device=x.device)
    v = torch.cat([x, pad], 1).view(rows, -1, BLOCK)
    amax = v.abs().amax(2, keepdim=True).clamp_min(448 * 2.0 ** -126)
    t = v.double() * 448.0 / amax.double()
    exponent = torch.frexp(t)[1].clamp_min(-5)  # t < 2^exponent; below 2^-6 the step stays
    step = torch.ldexp(torch.ones_like(t), exponent - 4)
    q = (torch.round(t / step) * step).float()
    return (q * (amax / 448.0)).view(rows, -1)[:, :k]


def _blocks(s, n, k):
    """Scales of the blocks, one for each weight: [.., n, k]."""
    return s.repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k]


def _plain_product(s):
    c = s["case"]
    x = s["x"].float()
    if c["source"] == "silu":
        x = x / (1 + torch.exp(-x)) * s["up"].float()
    x = _plain_quant(x)
    if c["source"] == "tokens":
        x = x[torch.div(s["sorted_ids"], c["top_k"], rounding_mode="floor").long()]
    out = torch.empty((c["rows"], c["n_out"]), dtype=_TORCH[c["dtype"]], device=DEVICE)
    spans = s["spans"]
    for e in range(len(spans) - 1):  # one product for each expert that holds rows
        if spans[e] == spans[e + 1]:
            continue
        w = s["w"][e].float() * _blocks(s["w_scales"][e], *s["w"][e].shape)
        out[spans[e]:spans[e + 1]] = torch.matmul(
            x[spans[e]:spans[e + 1]], w if c["transposed"] else w.t()).to(out.dtype)
    return out


def _plain_layer(s):
    c = s["case"]
    t, k, dim, h = c["tokens"], c["top_k"], c["dim"], c["hidden"]
    lg = s["logits"].float()
    order = torch.sort(lg, dim=1, descending=True, stable=True).indices[:, :k]
    weights = torch.gather(torch.softmax(lg, 1), 1, order)
    if c["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    ids = order.reshape(-1)

    def chosen(name, n, m):
        w, sc = s[name]
        return w.view(torch.uint8)[ids].view(w.dtype).float() * _blocks(sc[ids], n, m)

    x = s["x"].float().repeat_interleave(k, 0).unsqueeze(2)
    gate = torch.matmul(chosen("gate", h, dim), x)
    act = gate / (1 + torch.exp(-gate)) * torch.matmul(chosen("up", h, dim), x)
    rows = torch.matmul(chosen("down", dim, h), act).view(t, k, dim)
    return ((rows * weights.unsqueeze(2)).sum(1).to(s["x"].dtype), order.to(torch.int32), weights)


def _plain_norm(s):
    c = s["case"]
    dt = s["residual"].dtype
    y, wx, wy = s["y"].float(), s["x_weight"], s["y_weight"]
    gate = torch.ones((), device=DEVICE) if s["gate"] is None else s["gate"].float()
    n_y = y
    if wy is not None:
        ry = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        n_y = y * ry * wy
    r = s["residual_scale"] * s["residual"].float() + s["y_scale"] * gate * n_y
    rr = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    if not c["backward"]:
        return r.to(dt), (r * rr * wx).to(dt)
    hat = r * rr
    d_x = s["d_x"].float()
    g = d_x * wx
    d_r = s["d_r"].float() + rr * (g - hat * (g * hat).mean(1, keepdim=True))
    d_gate = s["y_scale"] * d_r * n_y
    d_n = s["y_scale"] * d_r * gate
    d_y, d_wy = d_n, None
    if wy is not None:
        hat_y = y * ry
        d_wy = (d_n * hat_y).sum(0)
        g = d_n * wy
        d_y = ry * (g - hat_y * (g * hat_y).mean(1, keepdim=True))
    d_gate = {"none": None, "channel": d_gate.sum(0), "token": d_gate.sum(1, keepdim=True),
              "full": d_gate.to(dt)}[c["gate"]]
    return ((s["residual_scale"] * d_r).to(dt), d_y.to(dt), (d_x * hat).sum(0), d_wy, d_gate)


_OWN = {"product": _own_product, "layer": _own_layer, "norm": _own_norm}
_PLAIN = {"product": _plain_product, "layer": _plain_layer, "norm": _plain_norm}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _present(experts, top_k, tokens):
    """Experts that hold a row, on average over evenly drawn choices."""
    return experts * (1.0 - (1.0 - top_k / experts) ** tokens)


def work(case):
    es = _SIZE[case["dtype"]]
    if case["op"] == "product":
        rows, k, n = case["rows"], case["k_in"], case["n_out"]
        e = _present(case["experts"], case["top_k"], rows // case["top_k"]) if case["experts"] else 1
        read = {"tokens": rows // case["top_k"], "rows": rows, "silu": 2 * rows}[case["source"]]
        return {"bytes": int(e * (n * k + 4 * -(-n // BLOCK) * -(-k // BLOCK))
                             + (read * k + rows * n) * es),
                "flops": 2 * rows * n * k}
    if case["op"] == "layer":
        t, k, dim, h = case["tokens"], case["top_k"], case["dim"], case["hidden"]
        e = _present(case["experts"], k, t)
        return {"bytes": int(e * 3 * dim * h + 2 * t * dim * es + t * case["experts"] * es + 8 * t * k),
                "flops": 6 * t * k * dim * h}
    t, dim = case["tokens"], case["dim"]
    arrays = 6 if case["backward"] else 4
    gate = t * dim * es * (2 if case["backward"] else 1) if case["gate"] == "full" else 0
    return {"bytes": arrays * t * dim * es + gate + 4 * dim * (2 if case["backward"] else 1),
            "flops": (30 if case["backward"] else 10) * t * dim}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    d = _inputs(case, seed)
    return {"product": _exact_product, "layer": _exact_layer, "norm": _exact_norm}[case["op"]](case, d)


def _expand(w, scales):
    """Weights as float64, block after block."""
    out = w.double()
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            out[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= scales[i, j].double()
    return out


def _exact_quant(x):
    """Rows of float64 through the table of E4M3's values: the nearest one, and
    half way between two the one with the even code."""
    codes = torch.arange(127, dtype=torch.uint8, device=x.device)
    table = codes.view(torch.float8_e4m3fn).double()
    middle = (table[1:] + table[:-1]) / 2
    out = torch.empty_like(x)
    for lo in range(0, x.shape[1], BLOCK):
        v = x[:, lo:lo + BLOCK]
        top = v.abs().amax(1, keepdim=True).clamp_min(448 * 2.0 ** -126)
        t = v.abs() * 448.0 / top
        below = torch.searchsorted(middle, t)             # middle[i - 1] < t <= middle[i]
        tie = (below < 126) & (middle[below.clamp_max(125)] == t) & (below % 2 == 1)
        out[:, lo:lo + BLOCK] = torch.sign(v) * table[below + tie.long()] * (top / 448.0)
    return out


def _exact_product(c, d):
    x = d["x"].double()
    if c["source"] == "silu":
        x = x * torch.sigmoid(x) * d["up"].double()
    x = _exact_quant(x)
    if c["source"] == "tokens":
        x = x.repeat_interleave(c["top_k"], 0)[d["sorted_ids"].long()]
    parts = []
    for e in range(len(d["spans"]) - 1):
        w = _expand(d["w"][e], d["w_scales"][e])
        parts.append(x[d["spans"][e]:d["spans"][e + 1]] @ (w if c["transposed"] else w.t()))
    return torch.cat(parts)


def _exact_layer(c, d):
    t, k = c["tokens"], c["top_k"]
    lg = d["logits"].double()
    out = torch.zeros((t, c["dim"]), dtype=torch.float64, device=DEVICE)
    weights = torch.zeros((t, k), dtype=torch.float64, device=DEVICE)
    for i in range(t):
        left = sorted(range(c["experts"]), key=lambda e, row=lg[i].tolist(): (-row[e], e))[:k]
        p = torch.exp(lg[i] - lg[i].max())
        p = p / p.sum()
        w = p[left]
        weights[i] = w / w.sum() if c["renorm"] else w
        x = d["x"][i].double()
        for j, e in enumerate(left):
            full = {n: _expand(d[n][0][e], d[n][1][e]) for n in ("gate", "up", "down")}
            g = full["gate"] @ x
            out[i] += weights[i, j] * (full["down"] @ (g * torch.sigmoid(g) * (full["up"] @ x)))
    return out, None, weights


def _exact_norm(c, d):
    names = ["residual", "y", "x_weight", "y_weight", "gate"]
    v = {n: d[n].double().requires_grad_(c["backward"]) for n in names if d[n] is not None}
    block = v["y"]
    if c["post"]:
        block = block / torch.sqrt(block.pow(2).mean(1, keepdim=True) + EPS) * v["y_weight"]
    if c["gate"] != "none":
        block = block * v["gate"]
    r = v["residual"] * d["residual_scale"] + block * d["y_scale"]
    x = r / torch.sqrt(r.pow(2).mean(1, keepdim=True) + EPS) * v["x_weight"]
    if not c["backward"]:
        return r, x
    got = dict(zip(v, torch.autograd.grad([r, x], list(v.values()),
                                          [d["d_r"].double(), d["d_x"].double()])))
    return tuple(got.get(n) for n in names)
