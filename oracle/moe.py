"""Plain CPU oracle of routing, products grouped by expert and block-scaled E4M3 (tests only).

Each straight from its definition in include/awq4.h, in binary64, rounded to
binary32 only where the definition says so; no code is shared with the GPU
library.  Tensors are numpy arrays of values (16-bit types widened by the caller).
"""
from __future__ import annotations

import numpy as np

TOP32 = float(np.finfo(np.float32).max)
NIBBLE_OF_COLUMN = (0, 4, 1, 5, 2, 6, 3, 7)  # inverse of the order (0, 2, 4, 6, 1, 3, 5, 7)


# ------------------------------------------------------------------ routing

def choose(logits, k: int, renormalize: bool):
    """(experts [T, k], weights [T, k]) one token and one choice at a time."""
    T, E = logits.shape
    experts = np.full((T, k), -1, dtype=np.int64)
    weights = np.zeros((T, k))
    for t in range(T):
        can = {e: min(float(logits[t, e]), TOP32) for e in range(E) if logits[t, e] > -np.inf}
        if not can:
            continue
        m = max(can.values())
        left = dict(can)
        for j in range(min(k, len(can))):
            best = max(left.values())
            e = min(i for i, v in left.items() if v == best)
            del left[e]
            experts[t, j], weights[t, j] = e, np.exp(best - m)
        weights[t] /= weights[t].sum() if renormalize else sum(np.exp(v - m) for v in can.values())
    return experts, weights


def plan(experts, E: int):
    """(offsets [E + 1], rows [T k], places [T k]) by lists, expert after expert."""
    flat = np.asarray(experts).reshape(-1)
    offsets, rows = [0], []
    places = np.full(flat.size, -1, dtype=np.int64)
    for e in range(E):
        for s in np.flatnonzero(flat == e):
            places[s] = len(rows)
            rows.append(int(s))
        offsets.append(len(rows))
    return np.array(offsets), np.array(rows + [-1] * (flat.size - len(rows)), dtype=np.int64), places


def combine(y, weights, places):
    """(sum of weights y, sum of |weights y|) of each token."""
    T, k = weights.shape
    out, size = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            p = int(places[t * k + j])
            if 0 <= p < len(y):
                out[t] += weights[t, j] * y[p]
                size[t] += np.abs(weights[t, j] * y[p])
    return out, size


# ------------------------------------------------------------------ weights

def dequant(qweight, scales, qzeros, group: int):
    """[K, N] values of packed int32 [K, N/8] (zero points 8 where there are none)."""
    def columns(words):
        w = np.asarray(words).view(np.uint32).astype(np.uint64)
        out = np.empty((w.shape[0], w.shape[1] * 8))
        for c in range(8):
            out[:, c::8] = (w >> np.uint64(4 * NIBBLE_OF_COLUMN[c])) & np.uint64(15)
        return out
    q = columns(qweight)
    z = np.full_like(np.asarray(scales, dtype=np.float64), 8.0) if qzeros is None else columns(qzeros)
    return (q - np.repeat(z, group, 0)) * np.repeat(np.asarray(scales, dtype=np.float64), group, 0)


def grouped(x, matrices, offsets, rows, top: int):
    """({row: x . W}, {row: |x| . |W|}) for matrices [K, N] per expert."""
    y, size = {}, {}
    for e, w in enumerate(matrices):
        for r in range(offsets[e], offsets[e + 1]):
            v = x[r] if rows is None else x[rows[r] // top]
            y[r], size[r] = v @ w, np.abs(v) @ np.abs(w)
    return y, size


# ------------------------------------------------------------------ E4M3

def _e4m3_values():
    out = np.empty(127)
    for c in range(127):
        e, m = c >> 3, c & 7
        out[c] = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return out


E4M3 = _e4m3_values()  # the values of codes 0 .. 126, rising


def decode(codes):
    c = np.asarray(codes, dtype=np.uint8)
    assert not np.any((c & 127) == 127)
    return np.where(c & 128, -1.0, 1.0) * E4M3[c & 127]


def encode(v):
    """Codes of |v| <= 448 by search: the nearest value, of two as near the one whose code is even."""
    a = np.abs(np.asarray(v, dtype=np.float64))
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def block_quant(x):
    """(codes [M, K], scales [M, ceil(K / 128)] binary32) of finite values."""
    M, K = x.shape
    codes, scales = np.empty((M, K), dtype=np.uint8), np.empty((M, -(-K // 128)), dtype=np.float32)
    for b in range(scales.shape[1]):
        v = x[:, 128 * b:128 * b + 128].astype(np.float64)
        s = (np.abs(v).max(1) / 448).astype(np.float32)
        scales[:, b] = s
        live = s > 0
        q = (v / np.where(live, s, 1).astype(np.float64)[:, None]).astype(np.float32)
        codes[:, 128 * b:128 * b + 128] = np.where(live[:, None], encode(np.clip(q, -448, 448)), 0)
    return codes, scales


def block_values(codes, scales, row_block: int):
    """Values of codes [M, K] with scales for each row_block rows and 128 columns."""
    v = decode(codes)
    s = np.repeat(np.repeat(np.asarray(scales, dtype=np.float64), row_block, 0)[:v.shape[0]], 128, 1)[:, :v.shape[1]]
    return v * s
