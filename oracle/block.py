"""Plain CPU oracle of the operators around the linear layers (tests only).

RMS norm with the residual's addition, rotary positions, the paged key/value
cache in 4 bits and causal attention over it, each straight from its definition
in include/awq4.h: binary64 arithmetic, one step at a time, rounded to binary32
or the activation type exactly where the definition says so.  No code is shared
with the GPU library.  Tensors are numpy arrays: 16-bit values as their uint16
patterns (dtype "f16" or "bf16"), the cache as int32 words.
"""
from __future__ import annotations

import numpy as np

ORDER = (0, 2, 4, 6, 1, 3, 5, 7)  # nibble i of a word holds column 8j + ORDER[i]


def decode(bits: np.ndarray, dtype: str) -> np.ndarray:
    """16-bit patterns -> binary64 values."""
    b = np.asarray(bits, dtype=np.uint16)
    if dtype == "f16":
        return b.view(np.float16).astype(np.float64)
    with np.errstate(invalid="ignore"):  # (widening a signalling NaN)
        return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def encode(v: np.ndarray, dtype: str) -> np.ndarray:
    """binary32 values -> 16-bit patterns, to nearest even."""
    f = np.asarray(v).astype(np.float32)
    if dtype == "f16":
        with np.errstate(over="ignore"):
            return f.astype(np.float16).view(np.uint16)
    u = f.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(f), np.uint16(0x7FC0), r)


def fl32(v):
    return np.asarray(v, dtype=np.float64).astype(np.float32).astype(np.float64)


# ------------------------------------------------------------------ RMS norm

def rmsnorm(x, residual, weight, eps: float, dtype: str):
    """(h, y) patterns [M, K] of the definition of w4a8_rmsnorm_quant."""
    h = np.asarray(x, dtype=np.uint16)
    if residual is not None:
        h = encode(fl32(decode(h, dtype) + decode(residual, dtype)), dtype)
    hv = decode(h, dtype)
    mean = (hv * hv).sum(axis=1, keepdims=True) / hv.shape[1]
    v = fl32(mean + np.float64(np.float32(eps)))
    q = fl32(1.0 / fl32(np.sqrt(v)))
    y = encode(fl32(fl32(hv * q) * decode(weight, dtype)[None, :]), dtype)
    return h, y


# ------------------------------------------------------------------ rotation

def rotate(x, rope_rows, interleaved: bool, dtype: str):
    """x patterns [T, H, D] turned by rope_rows fp32 [T, rot] (cosines, then sines)."""
    v = decode(x, dtype)
    rot = rope_rows.shape[1]
    c = rope_rows[:, None, :rot // 2].astype(np.float64)
    s = rope_rows[:, None, rot // 2:].astype(np.float64)
    first = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    second = first + (1 if interleaved else rot // 2)
    a, b = v[..., first], v[..., second]
    out = np.array(x, dtype=np.uint16)
    out[..., first] = encode(fl32(fl32(a * c) - fl32(b * s)), dtype)
    out[..., second] = encode(fl32(fl32(b * c) + fl32(a * s)), dtype)
    return out


# ------------------------------------------------------------------ 4 bits

def quantise(x, dtype: str):
    """(codes [..., D], scale patterns [...], zero points [...]) of patterns [..., D]."""
    v = decode(x, dtype)
    finite = np.isfinite(v).all(axis=-1)
    v = np.where(finite[..., None], v, 0.0)
    lo = np.minimum(v.min(axis=-1), 0.0)
    hi = np.maximum(v.max(axis=-1), 0.0)
    sb = encode(fl32(fl32(hi - lo) / 15.0), dtype)
    s = decode(sb, dtype)
    live = s != 0
    d = np.where(live, s, 1.0)
    z = np.minimum(np.rint(fl32(-lo / d)), 15.0)
    c = np.clip(np.rint(fl32(v / d[..., None])) + z[..., None], 0, 15)
    c = np.where(live[..., None], c, 0).astype(np.int64)
    z = np.where(live, z, 0).astype(np.int64)
    sb = np.where(finite, sb, np.uint16(0x7C01 if dtype == "f16" else 0x7F81))
    return c, sb, z


def pack(codes):
    """[..., D] codes -> [..., D/8] words."""
    c = np.asarray(codes, dtype=np.uint64).reshape(*codes.shape[:-1], -1, 8)
    w = np.zeros(c.shape[:-1], dtype=np.uint64)
    for i, col in enumerate(ORDER):
        w |= c[..., col] << np.uint64(4 * i)
    return w.astype(np.uint32).view(np.int32)


def head_words(D: int, P: int) -> int:
    return P * (D // 4 + 2)


def word_at(kind: str, P: int, D: int, token: int, j: int = 0) -> int:
    """Index of a word among those of one page and head."""
    if kind == "k":
        return token * (D // 8) + j
    if kind == "v":
        return P * (D // 8) + (token // 4) * (D // 8) * 4 + j * 4 + token % 4
    return 2 * P * (D // 8) + (P if kind == "vm" else 0) + token


def store(cache, P: int, slots, k, v, dtype: str) -> None:
    """Quantise k, v patterns [T, Hkv, D] into cache words [pages, Hkv, W]."""
    pages, hkv, _ = cache.shape
    D = k.shape[2]
    kc, ks, kz = quantise(k, dtype)
    vc, vs, vz = quantise(v, dtype)
    kw, vw = pack(kc), pack(vc)
    for t, slot in enumerate(np.asarray(slots)):
        if slot < 0 or slot >= pages * P:
            continue
        page, tok = int(slot) // P, int(slot) % P
        for h in range(hkv):
            row = cache[page, h]
            for j in range(D // 8):
                row[word_at("k", P, D, tok, j)] = kw[t, h, j]
                row[word_at("v", P, D, tok, j)] = vw[t, h, j]
            row[word_at("km", P, D, tok)] = int(ks[t, h]) | int(kz[t, h]) << 16
            row[word_at("vm", P, D, tok)] = int(vs[t, h]) | int(vz[t, h]) << 16


def append(q, k, v, rope, positions, slots, cache, P: int, interleaved: bool, dtype: str):
    """awq_kv4_append on numpy arrays: returns the rotated q, writes the cache."""
    slots = np.array(slots, dtype=np.int64)
    if rope is not None:
        pos = np.asarray(positions)
        ok = (pos >= 0) & (pos < rope.shape[0])
        rows = rope[np.where(ok, pos, 0)]
        slots[~ok] = -1
        k = rotate(k, rows, interleaved, dtype)
        if q is not None:
            q = rotate(q, rows, interleaved, dtype)
            q[~ok, :, :rope.shape[1]] = 0x7E00 if dtype == "f16" else 0x7FC0
    store(cache, P, slots, k, v, dtype)
    return q


def unpack(words):
    w = np.asarray(words).view(np.uint32)
    c = np.empty((*w.shape, 8), dtype=np.int64)
    for i, col in enumerate(ORDER):
        c[..., col] = (w >> np.uint32(4 * i)) & 0xF
    return c.reshape(*w.shape[:-1], -1)


def page_values(cache, P: int, D: int, page: int, h: int, dtype: str):
    """(K, V, K scales, V scales) of one page and head: [P, D] twice, [P] twice, in binary64."""
    row = np.ascontiguousarray(cache[page, h])
    n = P * D // 8
    kc = unpack(row[:n].reshape(P, D // 8))
    vc = unpack(np.ascontiguousarray(row[n:2 * n].reshape(P // 4, D // 8, 4).transpose(0, 2, 1)).reshape(P, D // 8))
    out = []
    for c, meta in ((kc, row[2 * n:2 * n + P]), (vc, row[2 * n + P:])):
        u = np.ascontiguousarray(meta).view(np.uint32)
        s = decode((u & 0xFFFF).astype(np.uint16), dtype)
        out.append(((c - (u >> 16).astype(np.int64)[:, None]) * s[:, None], s))
    return out[0][0], out[1][0], out[0][1], out[1][1]


# ------------------------------------------------------------------ attention

def _rows(q, cache, P: int, tables, lens, cu_q, scale: float, window: int, dtype: str):
    """For every row of q that sees anything: (row, query head, the row's values, scores of the tokens it sees, their
    softmax weights, values, key scales and value scales)."""
    T, hq, D = q.shape
    pages, hkv, _ = cache.shape
    G = hq // hkv
    qv = decode(q, dtype)
    for b in range(len(lens)):
        r0, r1 = int(cu_q[b]), int(cu_q[b + 1])
        n = r1 - r0
        length = min(max(int(lens[b]), 0), tables.shape[1] * P)
        if n == 0:
            continue
        j = np.arange(length)
        ids = tables[b][j // P] if length else np.zeros(0, dtype=np.int64)
        there = (ids >= 0) & (ids < pages)
        for h in range(hkv):
            K, V = np.zeros((length, D)), np.zeros((length, D))
            ks, vs = np.zeros(length), np.zeros(length)
            for first in range(0, length, P):
                if not there[first]:
                    continue
                m = min(P, length - first)
                pk, pv, sk, sv = page_values(cache, P, D, int(ids[first]), h, dtype)
                K[first:first + m], V[first:first + m] = pk[:m], pv[:m]
                ks[first:first + m], vs[first:first + m] = sk[:m], sv[:m]
            for i in range(n):
                p = length - n + i
                seen = there & (j <= p)
                if window:
                    seen &= j > p - window
                if not seen.any():
                    continue
                for e in range(h * G, (h + 1) * G):
                    row = qv[r0 + i, e]
                    t = scale * (K[seen] @ row)
                    w = np.exp(t - t.max())
                    w /= w.sum()
                    yield r0 + i, e, row, t, w, V[seen], ks[seen], vs[seen]


def attention(q, cache, P: int, tables, lens, cu_q, scale: float, window: int, dtype: str):
    """(out, spread, unit): out [T, Hq, D] in binary64, and what an error bound needs: sum of p |v| (spread), and per row
    (sum of p s', scale * largest |s| * sum |q|, largest s') over the tokens that it sees, from the words of the cache."""
    out, spread, unit = np.zeros(q.shape), np.zeros(q.shape), np.zeros((*q.shape[:2], 3))
    for r, e, row, _, w, V, ks, vs in _rows(q, cache, P, tables, lens, cu_q, scale, window, dtype):
        out[r, e] = w @ V
        spread[r, e] = w @ np.abs(V)
        unit[r, e] = (w @ vs, scale * np.abs(ks).max() * np.abs(row).sum(), np.nanmax(vs))
    return out, spread, unit


def products(q, cache, P: int, tables, lens, cu_q, scale: float, window: int, dtype: str):
    """[T, Hq, 3]: over the tokens that a row sees, the largest p |s'|, their number, and the sum of p |s'|."""
    top = np.zeros((*q.shape[:2], 3))
    for r, e, _, _, w, _, _, vs in _rows(q, cache, P, tables, lens, cu_q, scale, window, dtype):
        top[r, e] = (w * np.abs(vs)).max(), len(w), w @ np.abs(vs)
    return top
