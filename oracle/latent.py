"""Position rotation and latent attention in float64: the definitions that the
library's rotating writes, absorbed and expanded attention are checked against."""
from __future__ import annotations

import numpy as np


def table(positions: int, size: int, base: float = 10000.0) -> np.ndarray:
    """cos_sin rows: size / 2 cosines, then as many sines, of p / base^(2 i / size)."""
    angle = np.arange(positions)[:, None] * base ** (-np.arange(0, size, 2) / size)
    return np.concatenate([np.cos(angle), np.sin(angle)], -1)


def rotate(x, cos_sin, positions, pairs: bool) -> np.ndarray:
    """x [T, ..., D] with its first n = cos_sin.shape[1] dims turned."""
    x = np.array(x, np.float64)
    n = cos_sin.shape[1]
    row = np.asarray(cos_sin, np.float64)[np.asarray(positions)]
    row = row.reshape(row.shape[:1] + (1,) * (x.ndim - 2) + (n,))
    c, s = row[..., :n // 2], row[..., n // 2:]
    ia, ib = (slice(0, n, 2), slice(1, n, 2)) if pairs else (slice(0, n // 2), slice(n // 2, n))
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def rms_norm(c, weight, eps: float) -> np.ndarray:
    c = np.asarray(c, np.float64)
    return c / np.sqrt((c * c).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def attend(q, k, v, scale: float, prior: int):
    """One head: rows of q at positions prior, prior + 1, ... over keys 0 ..; returns the
    output and sum_p w_p |v_p|, which error bounds go by."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    logits = q @ k.T * scale
    hidden = np.arange(len(k))[None] > prior + np.arange(len(q))[:, None]
    logits[hidden] = -np.inf
    w = np.exp(logits - logits.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    return w @ v, w @ np.abs(v)


def absorbed(q, cache, block_tables, seq_lens, query_start_loc, scale: float, latent: int):
    """q [T, H, W] over cache [NB, 16, W]; returns out and sum |.| [T, H, latent]."""
    q = np.asarray(q, np.float64)
    rows = np.asarray(cache, np.float64).reshape(-1, cache.shape[-1])
    out = np.full(q.shape[:2] + (latent,), np.nan)
    mag = out.copy()
    for r, s in enumerate(seq_lens):
        a, b = query_start_loc[r], query_start_loc[r + 1]
        pos = np.arange(s)
        k = rows[np.asarray(block_tables)[r, pos // 16].astype(np.int64) * 16 + pos % 16]
        for h in range(q.shape[1]):
            out[a:b, h], mag[a:b, h] = attend(q[a:b, h], k, k[:, :latent], scale, s - (b - a))
    return out, mag


def expanded(q, k_nope, k_rope, v, query_start_loc, kv_start_loc, scale: float):
    """Ragged attention over each head's own keys beside the shared part."""
    out = np.full(q.shape[:2] + (v.shape[-1],), np.nan)
    mag = out.copy()
    for r in range(len(query_start_loc) - 1):
        a, b = query_start_loc[r], query_start_loc[r + 1]
        ka, kb = kv_start_loc[r], kv_start_loc[r + 1]
        for h in range(q.shape[1]):
            k = np.concatenate([k_nope[ka:kb, h], k_rope[ka:kb]], -1)
            out[a:b, h], mag[a:b, h] = attend(q[a:b, h], k, v[ka:kb, h], scale, (kb - ka) - (b - a))
    return out, mag
