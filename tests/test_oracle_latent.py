"""Pins of oracle/latent.py (CPU)."""
import numpy as np
import pytest
import torch

from oracle import latent as O


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("n,d", [(16, 64), (64, 64), (48, 128)])
def test_rotation(pairs, n, d):
    rng = np.random.default_rng(n + d)
    x, tab = rng.standard_normal((5, 3, d)), O.table(40, n)
    pos = np.array([0, 7, 39, 7, 1])
    y = O.rotate(x, tab, pos, pairs)
    assert np.array_equal(y[0], x[0])                       # position 0: angles of 0
    assert np.array_equal(y[..., n:], x[..., n:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))  # a rotation keeps lengths
    # hand-worked: the first pair turns by the position itself
    i, j = (0, 1) if pairs else (0, n // 2)
    assert np.allclose(y[1, :, i], x[1, :, i] * np.cos(7) - x[1, :, j] * np.sin(7))
    assert np.allclose(y[1, :, j], x[1, :, j] * np.cos(7) + x[1, :, i] * np.sin(7))
    # products depend on the distance alone
    a, b = x[:1, :1, :n], x[1:2, :1, :n]
    dot = [float((O.rotate(a, tab, [p], pairs) * O.rotate(b, tab, [p + 4], pairs)).sum()) for p in (0, 11, 30)]
    assert np.allclose(dot, dot[0])


def test_attend_matches_torch():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 24)), rng.standard_normal((9, 24)), rng.standard_normal((9, 8))
    out, mag = O.attend(q, k, v, 0.3, 6)
    mask = torch.ones(3, 9, dtype=torch.bool).tril(6)
    want = torch.nn.functional.scaled_dot_product_attention(*(torch.from_numpy(x)[None] for x in (q, k, v)),
                                                            attn_mask=mask, scale=0.3)[0]
    assert np.allclose(out, want.numpy(), atol=1e-12)
    assert (mag >= np.abs(out) - 1e-12).all()


def test_absorbed_is_expanded():
    """The two forms are one attention: with keys c Wk and values c Wv, absorbing Wk into q and
    applying Wv to the output gives the expanded form's result."""
    rng = np.random.default_rng(1)
    heads, r, rope, d, seqs, qs = 3, 32, 8, 12, [21, 5], [4, 1]
    wk, wv = rng.standard_normal((2, heads, r, d))
    starts, kvs = np.cumsum([0] + qs), np.cumsum([0] + seqs)
    c, kr = rng.standard_normal((kvs[-1], r)), rng.standard_normal((kvs[-1], rope))
    q = rng.standard_normal((starts[-1], heads, d + rope))
    tables = np.array([[3, 0], [2, -1]])
    cache = np.full((4, 16, r + rope), np.nan)
    for i in range(2):
        pos = np.arange(seqs[i])
        cache[tables[i, pos // 16], pos % 16] = np.concatenate([c, kr], -1)[kvs[i]:kvs[i + 1]]
    kn, v = (np.einsum("tr,hrd->thd", c, w) for w in (wk, wv))
    want, _ = O.expanded(q, kn, kr, v, starts, kvs, 0.2)
    qa = np.concatenate([np.einsum("thd,hrd->thr", q[..., :d], wk), q[..., d:]], -1)
    got, _ = O.absorbed(qa, cache, tables, seqs, starts, 0.2, r)
    assert np.allclose(np.einsum("thr,hrd->thd", got, wv), want, atol=1e-10)


def test_rms_norm():
    c, w = np.array([[3.0, -4.0, 0.0, 0.0]]), np.array([1.0, 2.0, 1.0, 1.0])
    assert np.allclose(O.rms_norm(c, w, 0.0), [[3 / 2.5, -8 / 2.5, 0, 0]])
    assert np.allclose(O.rms_norm(c, w, 8.0 - 0.25), [[3 / 14 ** 0.5, -8 / 14 ** 0.5, 0, 0]])
