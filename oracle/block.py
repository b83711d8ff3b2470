"""64-bit oracle of the operators around the routed experts: rows sorted by
expert and back, 8-bit integer products, the norms around a block (plain numpy;
test infrastructure only, shares no code with the library)."""
from __future__ import annotations

import numpy as np

# ---------------------------------------------------------------------------
# rows sorted by expert, and back
# ---------------------------------------------------------------------------


def order(ids: np.ndarray, E: int):
    """(offsets [E + 1], place [T, k]) one pair after the other."""
    flat = np.asarray(ids).reshape(-1)
    place = np.empty(flat.size, np.int64)
    offsets = np.zeros(E + 1, np.int64)
    row = 0
    for e in range(E):
        offsets[e] = row
        for p in np.flatnonzero(flat == e):
            place[p] = row
            row += 1
    offsets[E] = row
    for p in np.flatnonzero((flat < 0) | (flat >= E)):
        place[p] = -1 - row
        row += 1
    return offsets.astype(np.int32), place.reshape(np.shape(ids)).astype(np.int32)


def sort(x: np.ndarray, ids: np.ndarray, E: int):
    """(xs, offsets, place); rows of no expert are zeros."""
    T, k = ids.shape
    offsets, place = order(ids, E)
    xs = np.zeros((T * k, x.shape[1]), x.dtype)
    for t in range(T):
        for j in range(k):
            if place[t, j] >= 0:
                xs[place[t, j]] = x[t]
    return xs, offsets, place


def _row(ys, at):
    return ys[at] if 0 <= at < len(ys) else np.zeros(ys.shape[1])


def unsort(ys, place, weights=None):
    """(y, sums of the terms' magnitudes)"""
    ys = np.asarray(ys, np.float64)
    T, k = place.shape
    y, size = np.zeros((T, ys.shape[1])), np.zeros((T, ys.shape[1]))
    for t in range(T):
        for j in range(k):
            term = (1.0 if weights is None else float(weights[t, j])) * _row(ys, place[t, j])
            y[t] += term
            size[t] += np.abs(term)
    return y, size


def unsort_grad(dy, ys, place, weights=None):
    """(d_ys, d_weights, sums of the magnitudes behind d_weights)"""
    dy, ys = np.asarray(dy, np.float64), np.asarray(ys, np.float64)
    T, k = place.shape
    d_ys, d_w, size = np.zeros_like(ys), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            at = place[t, j]
            if 0 <= at < len(ys):
                d_ys[at] = (1.0 if weights is None else float(weights[t, j])) * dy[t]
                d_w[t, j] = (dy[t] * ys[at]).sum()
                size[t, j] = np.abs(dy[t] * ys[at]).sum()
    return d_ys, d_w, size


# ---------------------------------------------------------------------------
# 8-bit integer products
# ---------------------------------------------------------------------------


def quantize(x: np.ndarray):
    """(codes int8 [M, K], scales float32 [M]); the float32 roundings of the
    definition are made by numpy's float32."""
    x = np.asarray(x, np.float32)
    codes, scales = np.zeros(x.shape, np.int8), np.full(x.shape[0], np.nan, np.float32)
    for m, row in enumerate(x):
        if np.isfinite(row).all():
            a = np.maximum(np.abs(row).max(), np.float32(2.0 ** -100))
            scales[m] = a / np.float32(127)
            codes[m] = np.rint(row * (np.float32(127) / a))
    return codes, scales


def int8_product(w_codes, w_scales, x_codes, x_scales) -> np.ndarray:
    """y float32 [M, N]: the exact sums and the definition's three roundings."""
    sums = x_codes.astype(np.float64) @ w_codes.astype(np.float64).T  # (below 2^53: exact)
    with np.errstate(invalid="ignore", over="ignore"):
        return sums.astype(np.float32) * (x_scales.astype(np.float32)[:, None] * w_scales.astype(np.float32)[None, :])


def int8_grouped(w_codes, w_scales, x_codes, x_scales, offsets) -> np.ndarray:
    y = np.zeros((len(x_codes), w_codes.shape[1]), np.float32)
    for e in range(len(w_codes)):
        part = slice(offsets[e], offsets[e + 1])
        y[part] = int8_product(w_codes[e], w_scales[e], x_codes[part], x_scales[part])
    return y


# ---------------------------------------------------------------------------
# the norms around a block
# ---------------------------------------------------------------------------


def block_norm(x, y=None, post=None, gate=None, nxt=None, alpha=1.0, beta=1.0, eps=1e-6):
    """(r, h) in float64"""
    x = np.asarray(x, np.float64)
    inv = lambda v: 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    r = x
    if y is not None:
        u = np.asarray(y, np.float64)
        if post is not None:
            u = u * inv(u) * np.asarray(post, np.float64)
        if gate is not None:
            u = u * np.asarray(gate, np.float64)
        r = alpha * x + beta * u
    return r, None if nxt is None else r * inv(r) * np.asarray(nxt, np.float64)


def block_norm_grad(x, y, dr, dh, post=None, gate=None, nxt=None, alpha=1.0, beta=1.0, eps=1e-6):
    """(dx, dy, d_post, d_gate, d_next) by the chain rule, one row at a time."""
    f = lambda v: None if v is None else np.asarray(v, np.float64)
    x, y, dr, dh, post, gate, nxt = map(f, (x, y, dr, dh, post, gate, nxt))
    T, n = x.shape
    dx, dy = np.zeros((T, n)), np.zeros((T, n))
    d_post, d_next = np.zeros(n), np.zeros(n)
    d_gate = None if gate is None else np.zeros(gate.shape)
    whole = None if gate is None else np.broadcast_to(gate, (T, n))

    def back(v, weight, out):
        """gradient of v s(v) weight by v, and by the weight"""
        s = 1.0 / np.sqrt((v * v).mean() + eps)
        g = out * weight
        return s * g - v * (s ** 3 / n) * (g @ v), out * v * s

    for t in range(T):
        d = np.zeros(n) if dr is None else dr[t].copy()
        r = block_norm(x[t], None if y is None else y[t], post, None if gate is None else whole[t], None, alpha, beta, eps)[0]
        if dh is not None:
            more, w = back(r, nxt, dh[t])
            d += more
            d_next += w
        dx[t] = alpha * d
        if y is None:
            continue
        u = y[t] if post is None else y[t] / np.sqrt((y[t] * y[t]).mean() + eps) * post
        d = beta * d
        if gate is not None:
            if gate.ndim == 1:
                d_gate += d * u
            elif gate.shape[1] == n:
                d_gate[t] = d * u
            else:
                d_gate[t, 0] = (d * u).sum()
            d = d * whole[t]
        if post is not None:
            d, w = back(y[t], post, d)
            d_post += w
        dy[t] = d
    return (dx, None if y is None else dy, None if post is None else d_post, d_gate,
            None if nxt is None else d_next)
