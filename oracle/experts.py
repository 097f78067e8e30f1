"""Oracle for the expert operators: the sort of (point, expert) pairs, rows taken
to the experts' order and back with weights, the distillation loss against a
teacher's top logits, and the per-cell networks on sorted rows; with their
gradients, all in fp64. Test infrastructure only."""
from __future__ import annotations

import numpy as np

from . import nerf


def sort(ids, n_experts):
    """offset [E + 1], order [kept] and pos (shape of ids): kept pairs by (expert, pair)."""
    flat = np.asarray(ids, dtype=np.int64).ravel()
    kept = np.nonzero((flat >= 0) & (flat < n_experts))[0]
    order = np.array(sorted(kept.tolist(), key=lambda p: (flat[p], p)), dtype=np.int64)
    pos = np.full(flat.size, -1, dtype=np.int64)
    pos[order] = np.arange(order.size)
    offset = np.array([int((flat[kept] < e).sum()) for e in range(n_experts + 1)]) \
        if n_experts <= 64 else np.searchsorted(flat[order], np.arange(n_experts + 1))
    return offset, order, pos.reshape(np.shape(ids))


def _w(pos, weights):
    w = np.ones(pos.shape) if weights is None else np.asarray(weights, dtype=np.float64)
    return np.where(pos >= 0, w, 0.0)


def dispatch(x, pos, weights, rows):
    """rows with rows[pos] = w x."""
    out = np.array(rows, dtype=np.float64)
    w = _w(pos, weights)
    for i, j in zip(*np.nonzero(pos >= 0)):
        out[pos[i, j]] = w[i, j] * np.asarray(x[i], dtype=np.float64)
    return out


def taken(rows, pos):
    """rows[pos] [n][k][width], 0 for dropped pairs."""
    r = np.asarray(rows, dtype=np.float64)
    return np.where((pos >= 0)[..., None], r[np.maximum(pos, 0)], 0.0)


def combine(rows, pos, weights):
    return (_w(pos, weights)[..., None] * taken(rows, pos)).sum(axis=1)


def dots(rows, x, pos):
    """<x_i, rows[pos_ij]> [n][k]: the weight gradient of dispatch and combine."""
    return (taken(rows, pos) * np.asarray(x, dtype=np.float64)[:, None]).sum(axis=2)


def distill(student, teacher, ids, temperature, scale=None):
    """(loss [n], grad [n][classes]) of one teacher's kept logits per row."""
    s = np.asarray(student, dtype=np.float64) / temperature
    n, e = s.shape
    scale = np.ones(n) if scale is None else np.asarray(scale, dtype=np.float64)
    loss, grad = np.zeros(n), np.zeros((n, e))
    for i in range(n):
        kept = [j for j in range(ids.shape[1]) if 0 <= ids[i, j] < e and teacher[i, j] != -np.inf]
        if not kept:
            continue
        y = np.array([teacher[i, j] for j in kept], dtype=np.float64) / temperature
        logp = y - y.max() - np.log(np.exp(y - y.max()).sum())
        p = np.exp(logp)
        logq = s[i] - s[i].max() - np.log(np.exp(s[i] - s[i].max()).sum())
        at = ids[i, kept]
        with np.errstate(invalid="ignore"):
            loss[i] = temperature ** 2 * np.where(p > 0, p * (logp - logq[at]), 0.0).sum()
        g = np.exp(logq)
        np.subtract.at(g, at, p)
        grad[i] = scale[i] * temperature * g
    return loss, grad


N_CELL = 3317


def cell_parts(w):
    """W1 [32][63], b1, W2 [32][32], b2, ws [32], bs, Wc [3][59], bc of one cell's blob."""
    w = np.asarray(w, dtype=np.float64)
    c = np.split(w, np.cumsum([2016, 32, 1024, 32, 32, 1, 177]))
    return c[0].reshape(32, 63), c[1], c[2].reshape(32, 32), c[3], c[4], c[5], c[6].reshape(3, 59), c[7]


def encodings(x, d):
    return (nerf.positional_encoding(np.asarray(x, dtype=np.float64), 10),
            nerf.positional_encoding(nerf.unit(np.asarray(d)), 4))


def cells_forward(x, d, offset, cell_w):
    """raw [n][4] = (r, g, b, sigma) before activations and hidden [n][64]; 0 behind offset[-1]."""
    px, pd = encodings(x, d)
    raw, hidden = np.zeros((len(px), 4)), np.zeros((len(px), 64))
    for c in range(len(cell_w)):
        r = slice(offset[c], offset[c + 1])
        w1, b1, w2, b2, ws, bs, wc, bc = cell_parts(cell_w[c])
        h1 = np.maximum(px[r] @ w1.T + b1, 0.0)
        h2 = np.maximum(h1 @ w2.T + b2, 0.0)
        raw[r, :3] = np.concatenate([h2, pd[r]], axis=1) @ wc.T + bc
        raw[r, 3] = h2 @ ws + bs
        hidden[r] = np.concatenate([h1, h2], axis=1)
    return raw, hidden


def cells_backward(x, d, offset, cell_w, hidden, d_raw):
    """grad [cells][3317] of sum(raw * d_raw), the hidden layers as given."""
    px, pd = encodings(x, d)
    h, g = np.asarray(hidden, dtype=np.float64), np.asarray(d_raw, dtype=np.float64)
    grad = np.zeros((len(cell_w), N_CELL))
    for c in range(len(cell_w)):
        r = slice(offset[c], offset[c + 1])
        w1, b1, w2, b2, ws, bs, wc, bc = cell_parts(cell_w[c])
        h1, h2, gc, gs = h[r, :32], h[r, 32:], g[r, :3], g[r, 3]
        g2 = (gc @ wc[:, :32] + gs[:, None] * ws) * (h2 > 0)
        g1 = (g2 @ w2) * (h1 > 0)
        grad[c] = np.concatenate([(g1.T @ px[r]).ravel(), g1.sum(0), (g2.T @ h1).ravel(), g2.sum(0),
                                  gs @ h2, [gs.sum()],
                                  (gc.T @ np.concatenate([h2, pd[r]], axis=1)).ravel(), gc.sum(0)])
    return grad
