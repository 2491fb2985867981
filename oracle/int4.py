"""4-bit KV-cache quantisation for the oracle.  TEST INFRASTRUCTURE ONLY.

For a token, kv head and group of 32 head dims x the cache holds an f16 scale s,
an f16 zero z and 32 codes c in 0 .. 15; a code stands for (c s + z) * scale:
  y = x / scale in float32, saturated at +-16384 (infinities too);
  z = f16(min y), s = f16((max y - min y) / 15), in float32, ties to even;
  c = round((y - z) / s) clamped to 0 .. 15, ties to even; 0 where s is 0;
a group that holds a NaN has s = z = NaN.
A page (16-token block, kv head) of D = head_size has 8 D bytes of codes and 2 D
of parameters; where each code lies is spelled out per element below.

Written from that definition, element by element, apart from the CUDA path.
"""
from __future__ import annotations

import numpy as np

LIMIT = 16384.0
GROUP = 32
BLOCK = 16


def quantise(x, scale: float):
    """(codes uint8 [..., D], s f16 [..., D/32], z f16 [..., D/32]) of x."""
    y = np.asarray(x, np.float32) / np.float32(scale)
    y = np.where(np.isnan(y), y, np.clip(y, -LIMIT, LIMIT)).astype(np.float32)
    y = y.reshape(*y.shape[:-1], -1, GROUP)
    bad = np.isnan(y).any(-1)
    y = np.where(bad[..., None], np.float32(0), y)
    lo, hi = y.min(-1), y.max(-1)
    z = lo.astype(np.float16)
    s = ((hi - lo) / np.float32(15)).astype(np.float16)
    zf, sf = z.astype(np.float64)[..., None], s.astype(np.float64)[..., None]
    c = np.clip(np.rint((y.astype(np.float64) - zf) / np.where(sf > 0, sf, 1.0)), 0, 15)
    c = np.where(sf > 0, c, 0).astype(np.uint8)
    nan = np.float16(np.nan)
    return c.reshape(*c.shape[:-2], -1), np.where(bad, nan, s), np.where(bad, nan, z)


def k_place(t: int, d: int, D: int):
    """(byte, nibble) of dim d of token t in a K page."""
    g, r = divmod(d, GROUP)
    return t * (D // 2) + (r // 8) * (D // 8) + g * 4 + (r % 8) // 2, d % 2


def v_place(t: int, d: int, D: int):
    e, r = divmod(d, D // 8)
    return (t // 8) * 4 * D + e * (D // 2) + (t % 8) // 2 * (D // 8) + r // 4 * 4 + t % 2 * 2 + r % 4 // 2, d % 2


def k_param(t: int, g: int, D: int):
    """Bytes of s and z of group g of token t in a K page."""
    at = 8 * D + t * (D // 8) + 2 * g
    return at, at + D // 16


def v_param(t: int, g: int, D: int):
    at = 8 * D + 64 * g + 16 * ((t % 8) // 2) + 4 * (t // 8) + 2 * (t % 2)
    return at, at + 8


def _maps(is_v: bool, D: int):
    place, param = (v_place, v_param) if is_v else (k_place, k_param)
    at = np.array([[place(t, d, D) for d in range(D)] for t in range(BLOCK)])    # [16, D, 2]
    par = np.array([[param(t, g, D) for g in range(D // GROUP)] for t in range(BLOCK)])
    return at[..., 0], at[..., 1], par


def _f16_bytes(x):
    return np.ascontiguousarray(x, np.float16)[..., None].view(np.uint8)


def _put(pages, t: int, c, s, z, maps) -> None:
    """Write row t of pages [..., 10 D]: codes [..., D], parameters [..., D/32]."""
    byte, nib, par = maps
    for n in (0, 1):
        dims = np.nonzero(nib[t] == n)[0]
        old = pages[..., byte[t, dims]]
        pages[..., byte[t, dims]] = (old & (0xF0 if n == 0 else 0x0F)) | (c[..., dims] << (4 * n))
    for j, v in ((0, s), (1, z)):
        raw = _f16_bytes(v)
        pages[..., par[t, :, j]], pages[..., par[t, :, j] + 1] = raw[..., 0], raw[..., 1]


def store(cache, x, slot_mapping, scale: float, is_v: bool) -> np.ndarray:
    """A copy of the cache [NB, H, 10 D] with token t's rows x[t] quantised into
    slot slot_mapping[t]; negative slots are skipped."""
    out = np.array(cache, np.uint8, copy=True)
    maps = _maps(is_v, out.shape[-1] // 10)
    c, s, z = quantise(x, scale)
    for i, slot in enumerate(np.asarray(slot_mapping, np.int64)):
        if slot >= 0:
            _put(out[slot // BLOCK], int(slot) % BLOCK, c[i], s[i], z[i], maps)
    return out


def pack(x, scale: float, is_v: bool) -> np.ndarray:
    """The cache [NB, H, 10 D] that holds x [NB, 16, H, D] quantised."""
    x = np.asarray(x)
    nb, _, h, d = x.shape
    out = np.zeros((nb, h, 10 * d), np.uint8)
    maps = _maps(is_v, d)
    for t in range(BLOCK):
        _put(out, t, *quantise(x[:, t], scale), maps)
    return out


def params(cache, is_v: bool):
    """s and z, f16 [NB, 16, H, D/32], of every token of a cache."""
    c = np.asarray(cache, np.uint8)
    D = c.shape[-1] // 10
    par = _maps(is_v, D)[2]
    def read(at):
        raw = np.stack([c[:, :, at], c[:, :, at + 1]], -1)                        # [NB, H, 16, groups, 2]
        return np.ascontiguousarray(raw).view(np.float16)[..., 0].transpose(0, 2, 1, 3)
    return read(par[..., 0]), read(par[..., 1])


def codes(cache, is_v: bool) -> np.ndarray:
    """uint8 [NB, 16, H, D] codes of a cache."""
    c = np.asarray(cache, np.uint8)
    byte, nib, _ = _maps(is_v, c.shape[-1] // 10)
    return ((c[:, :, byte] >> (4 * nib)) & 15).astype(np.uint8).transpose(0, 2, 1, 3)


def dequantise(cache, scale: float, is_v: bool) -> np.ndarray:
    """float64 values [NB, 16, H, D] of a whole cache."""
    s, z = (np.repeat(a.astype(np.float64), GROUP, axis=-1) for a in params(cache, is_v))
    return (codes(cache, is_v) * s + z) * float(scale)
