"""fp64 forms of the 8-bit products, the MoE layer of a few tokens and the norms
around a block. NumPy, from the definitions; test infrastructure only."""
from __future__ import annotations

import numpy as np

from . import moe


def e4m3_values() -> np.ndarray:
    """The values of the codes 0 .. 126 (0x7f is NaN; 0x80 .. 0xff negate them)."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))


def e4m3_decode(codes: np.ndarray) -> np.ndarray:
    table = np.append(e4m3_values(), np.nan)
    codes = np.asarray(codes, dtype=np.uint8)
    return np.where(codes & 0x80, -1.0, 1.0) * table[codes & 0x7f]


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """Codes of the nearest values, half way between two the even code; |v| <= 448."""
    table = e4m3_values()
    a = np.abs(np.asarray(v, dtype=np.float64))
    hi = np.searchsorted(table, a).clip(1, 126)       # table[hi - 1] < a <= table[hi]
    lo = hi - 1
    down, up = a - table[lo], table[hi] - a
    code = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a == 0, 0, code)
    return (code + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quantise(x: np.ndarray, width: int):
    """(codes [rows, width], scales [groups, rows], both as defined) of rows x;
    a group that is not finite has a NaN scale and codes of 0."""
    rows, k = x.shape
    v = np.zeros((rows, width))
    v[:, :k] = x
    v = v.reshape(rows, -1, 128)
    m = np.abs(v).max(2)
    bad = ~np.isfinite(m)
    m = np.maximum(np.where(bad, 1.0, m), 448 * 2.0 ** -126)
    codes = e4m3_round(np.where(bad[:, :, None], 0.0, v) * 448.0 / m[:, :, None])
    codes[bad] = 0
    scales = np.where(bad, np.nan, m / 448.0)
    return codes.reshape(rows, width), scales.T


def silu(v: np.ndarray) -> np.ndarray:
    with np.errstate(over="ignore"):
        return v / (1 + np.exp(-v))


def expand(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp64 weights [E, N, K] of codes and block scales."""
    E, N, K = codes.shape
    s = np.asarray(scales, dtype=np.float64)
    return e4m3_decode(codes) * s[:, np.arange(N) // 128][:, :, np.arange(K) // 128]


def rows_of(codes: np.ndarray, scales: np.ndarray, k: int) -> np.ndarray:
    """fp64 rows [rows, k] of a quantised matrix."""
    s = np.asarray(scales, dtype=np.float64)
    return e4m3_decode(codes[:, :k]) * s.T[:, np.arange(k) // 128]


def products(weights: np.ndarray, q: np.ndarray, offsets, sorted_ids, top_k: int, base: np.ndarray):
    """(out, magnitude): base with the rows of every span replaced; the magnitude
    is the sum of the products' absolute values (0 for the rows left)."""
    out, mag = np.array(base, dtype=np.float64), np.zeros(base.shape)
    n = out.shape[0]
    off = [0, n] if offsets is None else [int(v) for v in offsets]
    src = np.arange(n) if sorted_ids is None else \
        np.where(np.asarray(sorted_ids) >= 0, np.asarray(sorted_ids) // top_k, -1)
    for e in range(len(off) - 1):
        r = np.arange(max(off[e], 0), min(off[e + 1], n))
        r = r[(src[r] >= 0) & (src[r] < q.shape[0])]
        out[r] = q[src[r]] @ weights[e].T
        mag[r] = np.abs(q[src[r]]) @ np.abs(weights[e]).T
    return out, mag


def layer(x, logits, gate, up, down, top_k: int, renorm: bool):
    """(out, indices, weights, magnitude) of the MoE layer; gate, up, down are fp64
    [E, ...] weights."""
    x = np.asarray(x, dtype=np.float64)
    idx = moe.router_choice(logits, top_k)
    w = moe.router_weights(logits, idx, renorm)
    out = np.zeros((x.shape[0], down.shape[1]))
    mag = np.zeros_like(out)
    for t in range(x.shape[0]):
        for j in range(top_k):
            e = idx[t, j]
            g, u = gate[e] @ x[t], up[e] @ x[t]
            act = w[t, j] * silu(g) * u
            out[t] += down[e] @ act
            # what errors of a few units of the sums' magnitudes in g and u become
            ga, ua = np.abs(gate[e]) @ np.abs(x[t]), np.abs(up[e]) @ np.abs(x[t])
            spread = w[t, j] * (1.1 * ga * np.abs(u) + np.abs(silu(g)) * ua) + np.abs(act)
            mag[t] += np.abs(down[e]) @ spread
    return out, idx, w, mag


def block_norm(residual, y=None, x_weight=None, y_weight=None, gate=None, residual_scale=1.0,
               y_scale=1.0, offset=0.0, eps=1e-6):
    """(r, x): see mlora_block_norm."""
    def norm(v, w):
        n = v / np.sqrt((v * v).mean(1, keepdims=True) + eps)
        return n if w is None else n * (w + offset)

    r = residual_scale * residual
    if y is not None:
        n = y if y_weight is None else norm(y, y_weight)
        r = r + y_scale * (1.0 if gate is None else gate) * n
    return r, norm(r, x_weight)


def block_norm_gradient(residual, d_r, d_x, y=None, x_weight=None, y_weight=None, gate=None,
                        residual_scale=1.0, y_scale=1.0, offset=0.0, eps=1e-6):
    """Dict of the gradients of sum(d_r r + d_x x), by the formulas."""
    D = residual.shape[1]
    r, _ = block_norm(residual, y, x_weight, y_weight, gate, residual_scale, y_scale, offset, eps)
    R = 1 / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    h = r * R
    g = d_x * (1.0 if x_weight is None else x_weight + offset)
    d = d_r + R * (g - h * (g * h).sum(1, keepdims=True) / D)
    out = {"residual": residual_scale * d, "x_weight": (d_x * h).sum(0)}
    if y is None:
        return out
    gt = 1.0 if gate is None else gate
    if y_weight is None:
        n, d_n = y, y_scale * d * gt
        out["y"] = d_n
    else:
        Ry = 1 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
        v = y * Ry
        n, d_n = v * (y_weight + offset), y_scale * d * gt
        out["y_weight"] = (d_n * v).sum(0)
        u = d_n * (y_weight + offset)
        out["y"] = Ry * (u - v * (u * v).sum(1, keepdims=True) / D)
    if gate is not None:
        dg = y_scale * d * n
        out["gate"] = dg.sum(0) if np.ndim(gate) == 1 else \
            dg.sum(1, keepdims=True) if gate.shape[1] == 1 and D > 1 else dg
    return out
