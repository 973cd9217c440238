"""Top-k router with padded slots, balance loss and gradients (CPU oracle).

TEST INFRASTRUCTURE ONLY -- see the package docstring. Written token by token, to be read
against the definitions of moe_route, moe_route_backward and moe_combine_backward in the
library's header; floating-point values in FP64.
"""

from __future__ import annotations

import numpy as np


def slots(tokens: int, experts: int, topk: int, pad: int) -> int:
    """The most slots a routing can need: one partly filled unit per expert that can be hit."""
    n = tokens * topk
    worst = n + min(n, experts) * (pad - 1)
    return worst - worst % pad


def choose(logits, topk: int, valid=None):
    """(topk_idx (T, k) int32, weights (T, k) FP64)."""
    z = np.asarray(logits, np.float64)
    T, G = z.shape
    idx = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    for t in range(T):
        if valid is not None and not valid[t]:
            continue
        usable = [e for e in range(G) if z[t, e] > -np.inf]
        best = sorted(usable, key=lambda e: (-z[t, e], e))[:topk]
        if best:
            p = np.exp(z[t, best] - z[t, best[0]])
            idx[t, :len(best)] = best
            w[t, :len(best)] = p / p.sum()
    return idx, w


def plan(idx, experts: int, pad: int, total: int):
    """counts (G + 1), offsets (G + 1), row_index (total), slot_of (T, k) of chosen experts idx."""
    T, k = idx.shape
    counts = np.zeros(experts + 1, np.int32)
    members = [[] for _ in range(experts)]
    for t in range(T):
        for e in idx[t]:
            if e >= 0:
                members[e].append(t)
        counts[experts] += idx[t, 0] >= 0
    units = []
    for e in range(experts):
        counts[e] = len(members[e])
        units.append(-(-len(members[e]) // pad))
    spare = total // pad - sum(units)
    assert spare >= 0
    for i in range(spare):
        units[i % experts] += 1
    offsets = np.concatenate([[0], np.cumsum(units)]).astype(np.int64) * pad
    row_index = np.full(total, -1, np.int32)
    slot_of = np.full((T, k), -1, np.int64)
    for e in range(experts):
        for i, t in enumerate(members[e]):
            row_index[offsets[e] + i] = t
            slot_of[t, list(idx[t]).index(e)] = offsets[e] + i
    return counts, offsets, row_index, slot_of


def softmax(logits, routed) -> np.ndarray:
    z = np.asarray(logits, np.float64)
    p = np.zeros_like(z)
    for t in np.flatnonzero(routed):
        e = np.where(z[t] > -np.inf, np.exp(z[t] - np.nanmax(z[t])), 0.0)
        p[t] = e / e.sum()
    return p


def balance_loss(logits, idx, counts, coef: float) -> float:
    G, n = logits.shape[1], counts[-1]
    if n == 0:
        return 0.0
    p = softmax(logits, idx[:, 0] >= 0)
    return float(coef * G * np.sum(counts[:G] / counts[:G].sum() * p.sum(axis=0) / n))


def backward(logits, idx, w, counts, d_weights, d_loss, coef: float) -> np.ndarray:
    T, G = logits.shape
    w = np.asarray(w, np.float64)
    d = np.zeros((T, G))
    if d_weights is not None:
        dw = np.asarray(d_weights, np.float64)
        for t in range(T):
            on = idx[t] >= 0
            mean = np.sum(w[t, on] * dw[t, on])
            d[t, idx[t, on]] = w[t, on] * (dw[t, on] - mean)
    if d_loss is not None and counts[-1] > 0:
        p = softmax(logits, idx[:, 0] >= 0)
        c = d_loss * coef * G * counts[:G].astype(np.float64) / (counts[:G].sum() * float(counts[-1]))
        d += p * (c - (p @ c)[:, None])
    return d


def combine_backward(dy, o_slots, slot_of, w):
    """FP64 (d_o (S, H), padding rows zero; d_weights (T, k))."""
    dy, o = np.asarray(dy, np.float64), np.asarray(o_slots, np.float64)
    d_o, d_w = np.zeros_like(o), np.zeros(slot_of.shape)
    for t in range(slot_of.shape[0]):
        for j, s in enumerate(slot_of[t]):
            if 0 <= s < o.shape[0]:
                d_o[s] = float(w[t, j]) * dy[t]
                d_w[t, j] = dy[t] @ o[s]
    return d_o, d_w
