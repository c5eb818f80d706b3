"""8-bit rows, the norm ahead of them, products with 8-bit weights, and log probabilities (oracle; test infrastructure only).

Definitions: a row's norm is y = h / sqrt(mean(h^2) + eps) * (weight_offset + weight) with h = x + residual.  8-bit rows hold
e4m3 codes with one fp32 scale per 128 features: scale = max |y| (1 / 448), code = e4m3(y / scale) to nearest even; these are
whole decisions, so the product (with 1 / 448 rounded to fp32) and the division are taken in fp32 as the definition says.  Weights hold one scale per block of 128 x 128.
Log probabilities are of softmax(logits / T); an equal logit at a lower index ranks first.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
INV_TOP = np.float32(1.0) / np.float32(448.0)


def e4m3_table() -> np.ndarray:
    """fp64 value of every byte: sign, 4 bits of exponent (bias 7), 3 bits of mantissa; 0x7F and 0xFF are NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = np.nan if c & 0x7F == 0x7F else -v if c & 0x80 else v
    return out


TABLE = e4m3_table()


def decode(codes) -> np.ndarray:
    return TABLE[np.asarray(codes, dtype=np.uint8)]


def encode(x) -> np.ndarray:
    """Nearest e4m3 code, ties to the even mantissa, beyond 448 clamped, NaN to 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    mag = TABLE[:0x7F]  # ascending
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0)), 448.0)
    hi = np.minimum(np.searchsorted(mag, a), 0x7E)  # the first code at or above
    lo = np.maximum(hi - 1, 0)
    up, down = mag[hi] - a, a - mag[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    c = np.where(mag[hi] == a, hi, c)
    c = np.where(np.signbit(x), c | 0x80, c)
    return np.where(np.isnan(x), 0x7F, c).astype(np.uint8)


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def quantize(x):
    """(codes uint8 [rows, H], scale fp32 [rows, ceil(H / 128)]) of fp32 rows, group by group."""
    x = np.asarray(x, dtype=np.float32)
    rows, H = x.shape
    codes, scale = np.zeros((rows, H), np.uint8), np.zeros((rows, blocks(H)), np.float32)
    with np.errstate(all="ignore"):
        for j in range(blocks(H)):
            g = x[:, j * BLOCK:(j + 1) * BLOCK]
            s = np.abs(g).max(axis=1) * INV_TOP  # max keeps a NaN
            q = np.where(s[:, None] == 0, np.float32(0), g / s[:, None])
            codes[:, j * BLOCK:(j + 1) * BLOCK], scale[:, j] = encode(q), s
    return codes, scale


def add_rms_norm(x, weight, eps, residual=None, weight_offset=0.0):
    """(h, y) in fp64."""
    h = np.asarray(x, np.float64) + (0 if residual is None else np.asarray(residual, np.float64))
    with np.errstate(all="ignore"):
        return h, h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * (weight_offset + np.asarray(weight, np.float64))


def spread(codes, scale, rows_per_scale: int) -> np.ndarray:
    """fp64 values of e4m3 codes [n, k]: rows_per_scale 1 for rows, 128 for weights."""
    s = np.repeat(np.repeat(np.asarray(scale, np.float64), rows_per_scale, 0)[:codes.shape[0]], BLOCK, 1)[:, :codes.shape[1]]
    with np.errstate(all="ignore"):
        return decode(codes) * s


def matmul(a, a_scale, w, w_scale) -> np.ndarray:
    return spread(a, a_scale, 1) @ spread(w, w_scale, BLOCK).T


def logprobs(logits, targets=None, temperature=1.0, top_k=0):
    """dict(logp, rank, entropy, top_tokens, top_logp) of fp64 logits [rows, V]."""
    x = np.asarray(logits, np.float64)
    rows, V = x.shape
    got = dict(logp=np.full(rows, np.nan), rank=np.full(rows, -1), entropy=np.full(rows, np.nan),
               top_tokens=np.full((rows, top_k), -1), top_logp=np.full((rows, top_k), np.nan))
    for r in range(rows):
        m = x[r].max()
        if not np.isfinite(m):  # NaN, +infinity, or nothing but -infinity
            continue
        z = (x[r] - m) / temperature
        p = np.exp(z)
        total = p.sum()
        lp = z - np.log(total)
        p /= total
        got["entropy"][r] = -(p[p > 0] * lp[p > 0]).sum()
        order = np.lexsort((np.arange(V), -x[r]))
        got["top_tokens"][r], got["top_logp"][r] = order[:top_k], lp[order[:top_k]]
        t = -1 if targets is None else int(targets[r])
        if 0 <= t < V:
            got["logp"][r] = lp[t]
            got["rank"][r] = (x[r] > x[r, t]).sum() + (x[r, :t] == x[r, t]).sum()
    return got
