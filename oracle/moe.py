"""fp64 forms of the MoE layer's operators around the fold: the router's
choice and its gradient, the stable sort by expert, dispatch, the weighted
combine and its gradient, and products with 4-bit weights. Plain loops and
NumPy, from the definitions; test infrastructure only."""
from __future__ import annotations

import numpy as np


def router_choice(logits: np.ndarray, top_k: int) -> np.ndarray:
    """Indices of the top_k largest values of each row, ties to the lowest
    index, a NaN above every number, -0 equal to +0."""
    out = np.empty((logits.shape[0], top_k), dtype=np.int32)
    for t, row in enumerate(np.asarray(logits, dtype=np.float64)):
        key = np.where(np.isnan(row), np.inf, row)
        order = sorted(range(row.size), key=lambda e: (not np.isnan(row[e]), -key[e], e))
        out[t] = order[:top_k]
    return out


def router_weights(logits: np.ndarray, indices: np.ndarray, renorm: bool) -> np.ndarray:
    """Softmax probabilities of the chosen experts (over all experts, or over
    the chosen ones); 0 for a row with nothing but -inf."""
    lg = np.asarray(logits, dtype=np.float64)
    w = np.zeros(indices.shape)
    for t in range(lg.shape[0]):
        top = lg[t].max()
        if top == -np.inf:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            ex = np.exp(lg[t] - top)
            chosen = ex[indices[t]]
            w[t] = chosen / (chosen.sum() if renorm else ex.sum())
    return w


def router_gradient(logits: np.ndarray, indices: np.ndarray, d_weights: np.ndarray,
                    renorm: bool) -> np.ndarray:
    """d/dlogits of sum(d_weights * weights) for fixed indices."""
    lg = np.asarray(logits, dtype=np.float64)
    out = np.zeros_like(lg)
    for t in range(lg.shape[0]):
        live = [e for e in (indices[t] if renorm else range(lg.shape[1]))]
        top = lg[t, live].max()
        if top == -np.inf:
            continue
        p = np.zeros(lg.shape[1])
        p[live] = np.exp(lg[t, live] - top)
        p /= p.sum()
        dw = np.zeros(lg.shape[1])
        dw[indices[t]] = d_weights[t]
        out[t] = p * (dw - (dw * p).sum())
    return out


def sort_by_expert(ids: np.ndarray, n_experts: int):
    """(expert_offsets, sorted_ids, slot_rows) of the stable sort; ids outside
    [0, n_experts) dropped."""
    buckets = [[] for _ in range(n_experts)]
    for i, e in enumerate(ids.tolist()):
        if 0 <= e < n_experts:
            buckets[e].append(i)
    offsets = np.zeros(n_experts + 1, dtype=np.int32)
    offsets[1:] = np.cumsum([len(b) for b in buckets])
    flat = [i for b in buckets for i in b]
    sorted_ids = np.full(ids.size, -1, dtype=np.int32)
    sorted_ids[: len(flat)] = flat
    slot_rows = np.full(ids.size, -1, dtype=np.int32)
    slot_rows[flat] = np.arange(len(flat), dtype=np.int32)
    return offsets, sorted_ids, slot_rows


def dispatch(x: np.ndarray, sorted_ids: np.ndarray, top_k: int) -> np.ndarray:
    rows = np.zeros((sorted_ids.size, x.shape[1]), dtype=x.dtype)
    live = sorted_ids >= 0
    rows[live] = x[sorted_ids[live] // top_k]
    return rows


def _places(n_tokens, top_k, slot_rows, n_rows):
    rows = np.arange(n_tokens * top_k) if slot_rows is None else np.asarray(slot_rows)
    rows = np.where((rows >= 0) & (rows < n_rows), rows, -1)
    return rows.reshape(n_tokens, top_k)


def combine(rows: np.ndarray, n_tokens: int, top_k: int, weights, slot_rows):
    """(out, magnitude): the weighted sums and the sums of absolute values."""
    rows = np.asarray(rows, dtype=np.float64)
    at = _places(n_tokens, top_k, slot_rows, rows.shape[0])
    out = np.zeros((n_tokens, rows.shape[1]))
    mag = np.zeros_like(out)
    for t in range(n_tokens):
        for j in range(top_k):
            if at[t, j] >= 0:
                w = 1.0 if weights is None else float(weights[t, j])
                out[t] += w * rows[at[t, j]]
                mag[t] += abs(w) * np.abs(rows[at[t, j]])
    return out, mag


def combine_gradient(d_out: np.ndarray, rows: np.ndarray, top_k: int, weights, slot_rows):
    """(d_rows, d_weights, magnitude of d_weights)."""
    d_out = np.asarray(d_out, dtype=np.float64)
    rows = np.asarray(rows, dtype=np.float64)
    n_tokens = d_out.shape[0]
    at = _places(n_tokens, top_k, slot_rows, rows.shape[0])
    d_rows = np.zeros_like(rows)
    d_w = np.zeros((n_tokens, top_k))
    mag = np.zeros_like(d_w)
    for t in range(n_tokens):
        for j in range(top_k):
            r = at[t, j]
            if r >= 0:
                d_rows[r] = (1.0 if weights is None else float(weights[t, j])) * d_out[t]
                d_w[t, j] = d_out[t] @ rows[r]
                mag[t, j] = np.abs(d_out[t]) @ np.abs(rows[r])
    return d_rows, d_w, mag


def w4_weights(q: np.ndarray, scales: np.ndarray, zeros, k_in: int, group: int) -> np.ndarray:
    """fp64 weights [E, N, K] of packed bytes (k even in the low half)."""
    v = np.empty(q.shape[:2] + (k_in,))
    v[..., 0::2] = q & 15
    v[..., 1::2] = q >> 4
    g = np.arange(k_in) // group
    z = 8.0 if zeros is None else (np.asarray(zeros) & 15).astype(np.float64)[..., g]
    return (v - z) * np.asarray(scales, dtype=np.float64)[..., g]


def w4_products(weights: np.ndarray, x: np.ndarray, ids, top_k: int, x_by_row: bool,
                n_rows: int) -> np.ndarray:
    """The products (weights: from w4_weights; with |weights| and |x| bounds,
    the sums of their absolute values)."""
    x = np.asarray(x, dtype=np.float64)
    out = np.zeros((n_rows, weights.shape[1]))
    for r in range(n_rows):
        e = 0 if ids is None else int(ids[r])
        if 0 <= e < weights.shape[0]:
            out[r] = weights[e] @ x[r if x_by_row else r // top_k]
    return out
