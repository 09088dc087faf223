"""What surrounds the verification step, in plain fp64 numpy (oracle).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Ancestor bits of token trees; rotary positions; the 8-bit entry format; the
attention of a verify pass; the rules on the logits.  Each function is the
definition, row by row, and shares nothing with the CUDA path.
"""

from __future__ import annotations

import numpy as np

TAIL = 16  # bytes after an 8-bit entry's codes: its fp32 scale, then zeros


def ancestors(parent, n):
    """(bits [N+1, N+1] bool, depth [N+1]) of one tree; rows past n are empty."""
    N = len(parent)
    bits, depth = np.zeros((N + 1, N + 1), bool), np.zeros(N + 1, np.int32)
    for i in range(min(n, N) + 1 if n >= 0 else 0):
        j = i
        while True:
            bits[i, j] = True
            if j == 0:
                break
            j = int(parent[j - 1])
        depth[i] = bits[i].sum() - 1
    return bits, depth


def pack(bits, words=None):
    """[..., n] bool -> [..., words] uint32, bit j of word w = column 32 w + j."""
    n = bits.shape[-1]
    words = -(-n // 32) if words is None else words
    full = np.zeros(bits.shape[:-1] + (words * 32,), np.uint64)
    full[..., :n] = bits
    full = full.reshape(bits.shape[:-1] + (words, 32))
    return (full << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)


def rotate(x, cos, sin, pairs):
    """x [..., D] fp64, cos / sin [..., rot/2]: the first rot columns rotated."""
    x = np.array(x, np.float64)
    half = cos.shape[-1]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    x1, x2 = x[..., a].copy(), x[..., b].copy()
    x[..., a], x[..., b] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return x


def e4m3_value(code):
    """Sign, 4 exponent bits (bias 7), 3 fraction bits; code 127 is NaN, no infinity."""
    c = np.asarray(code).astype(np.int64)
    e, f = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def e4m3_scale(x):
    """Smallest power of two s with max|x| <= 448 s over the last axis (1 for zeros, as
    keys are stored; values that are all zeros have 2^-126)."""
    big = np.nanmax(np.abs(np.asarray(x, np.float64)), axis=-1)
    out = np.ones_like(big)
    for at in np.ndindex(big.shape):
        if big[at] > 0:
            s = -126
            while big[at] > 448 * 2.0 ** s:
                s += 1
            out[at] = 2.0 ** s
    return out


def e4m3_round(y):
    """Nearest representable value, ties to even fractions, saturating."""
    y = np.asarray(y, np.float64)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.clip(np.rint(y / step) * step, -448, 448)


def decode(rows, fmt, D):
    """Entry rows -> fp64 values.  rows: uint8 [..., D + 16] (e4m3) or numbers [..., D]."""
    if fmt != "e4m3":
        return np.asarray(rows, np.float64)
    scale = np.ascontiguousarray(rows[..., D:D + 4]).view(np.float32)[..., 0].astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        return e4m3_value(rows[..., :D]) * scale[..., None]


def attend(q, K, V, seen, scale):
    """One row over its keys: q [D], K, V [n, D], seen [n] -> (o, sum p |v|, sum p |score parts|).

    Only what is seen enters; a row that sees nothing is zero."""
    idx = np.flatnonzero(seen)
    D = q.shape[0]
    if idx.size == 0:
        return np.zeros(D), np.zeros(D), 0.0
    K, V = K[idx], V[idx]
    s = (K @ q) * scale
    size = (np.abs(K) @ np.abs(q)).max() * abs(scale)
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ V, p @ np.abs(V), size


def adjust(l, V, counts, rep, pres, freq, bias, allowed):
    """One row of logits [V] -> adjusted fp64, and the size of what was added up."""
    l = np.array(l, np.float64)
    size = np.abs(l)
    hit = counts > 0
    y = np.where(l > 0, l / rep, l * rep)
    size = np.where(hit, np.abs(y) + np.abs(freq * counts) + abs(pres), size)
    l = np.where(hit, y - freq * counts - pres, l) + bias
    size = size + np.abs(bias)
    if allowed is not None:
        l[~allowed] = -np.inf
    return l, size
