"""64-bit oracle of expert selection, its gradient and the 8-bit products
(plain numpy; test infrastructure only, shares no code with the library)."""
from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# expert selection
# ---------------------------------------------------------------------------


def scores(logits: np.ndarray, scoring: str) -> np.ndarray:
    """Scores of one row of logits (float64); a sigmoid below float32's
    smallest normal number is zero, as the definition's float32 score is."""
    l = np.asarray(logits, np.float64)
    if scoring == "sigmoid":
        s = 1.0 / (1.0 + np.exp(-np.clip(l, -700, None)))
        return np.where(s < 2.0 ** -126, 0.0, s)
    top = l.max()
    if top == -np.inf:
        return np.zeros_like(l)
    e = np.exp(l - top)
    return e / e.sum()


def _best(values, count):
    """Indices of the `count` largest values above -inf, equal ones by index."""
    order = sorted((i for i in range(len(values)) if values[i] != -np.inf), key=lambda i: (-values[i], i))
    return order[:count]


def router(logits, k, scoring, bias=None, n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0):
    """(ids [T, k], weights [T, k]) by the definition, one row at a time."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    ids = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k), np.float64)
    for t in range(T):
        l = logits[t]
        if np.isnan(l).any() or (bias is not None and np.isnan(bias).any()) or (
                scoring == "softmax" and (l == np.inf).any()):
            weights[t] = np.nan
            continue
        s = scores(l, scoring)
        c = l.copy() if bias is None else np.where(l == -np.inf, -np.inf, s + np.asarray(bias, np.float64))
        if n_group > 1:
            per = E // n_group
            worth = np.full(n_group, -np.inf)
            for g in range(n_group):
                member = c[g * per:(g + 1) * per]
                value = s[g * per:(g + 1) * per] if bias is None and group_top == 2 else member
                value = np.sort(value[member != -np.inf])[::-1]
                if value.size:
                    worth[g] = value[:group_top].sum()
            stay = _best(worth, topk_group)
            for g in range(n_group):
                if g not in stay:
                    c[g * per:(g + 1) * per] = -np.inf
        chosen = _best(c, k)
        if not chosen:
            continue
        d = s[chosen].sum() if renorm else 1.0
        ids[t] = chosen[0]
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = scale * s[chosen] / d if d > 0 else 0.0
    return ids, weights


def router_gap(logits, k, scoring, bias, n_group=1, topk_group=1, group_top=1) -> float:
    """Smallest nonzero distance between two values that a choice compares,
    over all rows (finite ones): how far rounding may go before it changes an id."""
    logits = np.asarray(logits, np.float64)
    E = logits.shape[1]
    least = np.inf
    for l in logits:
        s = scores(l, scoring)
        c = l if bias is None else s + np.asarray(bias, np.float64)
        sets = [c[np.isfinite(c)]]
        if n_group > 1:
            v = s if bias is None and group_top == 2 else c
            sets.append(np.sort(v.reshape(n_group, E // n_group))[:, ::-1][:, :group_top].sum(1))
        for v in sets:
            d = np.diff(np.sort(v))
            d = d[d > 0]
            if d.size:
                least = min(least, d.min())
    return least


def router_grad(logits, ids, d_weights, scoring, renorm, scale):
    """d_logits [T, E] from the chain rule, the choice held fixed."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        slots = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E and (j == 0 or ids[t, j] != ids[t, 0])]
        if not slots:
            continue
        at = ids[t, slots]
        s = scores(logits[t], scoring)
        g = scale * np.asarray(d_weights, np.float64)[t, slots]
        ds = np.zeros(E)
        if renorm:
            d = s[at].sum()
            if d == 0:
                continue
            ds[at] = (g - (g * s[at]).sum() / d) / d
        else:
            ds[at] = g
        out[t] = ds * s * (1 - s) if scoring == "sigmoid" else s * (ds - (ds * s).sum())
    return out


# ---------------------------------------------------------------------------
# 8-bit products
# ---------------------------------------------------------------------------


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes."""
    v = np.empty(256)
    for code in range(256):
        sign, e, m = (-1.0 if code & 0x80 else 1.0), (code >> 3) & 15, code & 7
        v[code] = sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        if code & 0x7F == 0x7F:
            v[code] = np.nan
    return v


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """Codes nearest to x (|x| <= 464), ties to the even code."""
    x = np.asarray(x, np.float64)
    table = e4m3_values()[:127]  # codes 0 .. 126: 0 .. 448, increasing
    a = np.abs(x)
    hi = np.clip(np.searchsorted(table, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up = table[hi] - a
    down = a - table[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(np.isnan(x), 0x7F, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def quantize(x: np.ndarray):
    """(codes uint8 [M, K], scales float32 [M, ceil(K / 128)]) of finite x;
    the float32 roundings of the definition are made by numpy's float32."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    nb = -(-K // BLOCK)
    codes = np.zeros((M, K), np.uint8)
    sc = np.zeros((M, nb), np.float32)
    for b in range(nb):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        a = np.maximum(np.abs(v).max(1), np.float32(2.0 ** -100))
        r = np.float32(E4M3_MAX) / a
        codes[:, b * BLOCK:(b + 1) * BLOCK] = to_e4m3(v * r[:, None])
        sc[:, b] = a / np.float32(E4M3_MAX)
    return codes, sc


def linear(w_codes, w_scales, x_codes, x_scales) -> np.ndarray:
    """y [M, N] (float64) from codes [N, K] / [M, K] and their block scales."""
    table = e4m3_values()
    N, K = w_codes.shape
    y = np.zeros((x_codes.shape[0], N))
    for b in range(-(-K // BLOCK)):
        part = slice(b * BLOCK, (b + 1) * BLOCK)
        d = table[x_codes[:, part]] @ table[w_codes[:, part]].T
        sw = np.asarray(w_scales, np.float64)[np.arange(N) // BLOCK, b]
        y += d * np.asarray(x_scales, np.float64)[:, b:b + 1] * sw[None, :]
    return y
