"""Softmax references that move between key tiles, under a sharp bound: keys stand on stairs of about 2^9.5 (in
weight), a single key on the last of them, so that the hundreds of keys before it keep a share of every row that
a wrong factor of the move would show in.  Rows feel the stairs by 0.5, 1 or 1.3, so some columns move where
their neighbours do not."""
import numpy as np
import pytest
import torch

import paged_kv_attention_04_gb300 as P
from latent_cases import Step, bound, check
from test_gpu_expanded import Prompts

BF16 = torch.bfloat16
STAIR = 9.5 * np.log(2.0)
SCALE = 2.0 ** -4


def stairs(n, tile, stairs_at, rng, last=None):
    """Logit of each of n keys: the stairs begin with the tiles of stairs_at, the last is a single key of its tile
    (below key `last`)."""
    x = np.zeros(n)
    for t in stairs_at[:-1]:
        x[t * tile:] += STAIR
    t = stairs_at[-1]
    end = min((t + 1) * tile, n if last is None else last)
    x[rng.integers(t * tile, end)] += STAIR
    return x


def absorbed_step(heads, latent, q_lens, seq_lens, seed):
    """A request's tiles of 64 keys: a stair after the first third, the single key in one of the last tiles that
    every row of the request sees."""
    step = Step(heads, latent, q_lens, seq_lens, BF16, seed=seed, scale=SCALE)
    rng = np.random.default_rng(seed)
    step.q = (step.q * 0.25).to(BF16)
    step.q[..., latent] = torch.from_numpy(rng.choice([0.5, 1.0, 1.3], step.q.shape[:2])).to(BF16)
    for r, n in enumerate(step.seq_lens):
        n = int(n)
        seen = n - int(step.q_lens[r]) + 1  # keys that the first row sees
        tiles = -(-seen // 64)
        at = [tiles - 1 - int(rng.integers(0, min(3, tiles)))]
        if at[0] > 6:
            at = [max(1, at[0] - 5)] + at
        pos = np.arange(n)
        x = torch.from_numpy(stairs(n, 64, at, rng, seen) / SCALE).to(BF16)
        step.cache[step.tables[r, pos // 16], pos % 16, latent] = x
    return step


def expanded_step(heads, size, q_lens, seq_lens, seed):
    step = Prompts(heads, size, q_lens, seq_lens, seed=seed, scale=SCALE)
    rng = np.random.default_rng(seed)
    step.q = (step.q * 0.25).to(BF16)
    step.q[..., size] = torch.from_numpy(rng.choice([0.5, 1.0, 1.3], step.q.shape[:2])).to(BF16)
    for r, n in enumerate(step.seq_lens):
        seen = int(n - step.q_lens[r]) + 1
        tiles = -(-seen // 80)
        at = [tiles - 1 - int(rng.integers(0, min(3, tiles)))]
        if at[0] > 6:
            at = [at[0] - 5] + at
        a = int(step.kv_starts[r])
        step.rope[a:a + int(n), 64] = torch.from_numpy(stairs(int(n), 80, at, rng, seen) / SCALE).to(BF16)
    return step


WHOLE = [(16, [1] * 24, list(range(129, 385, 11))), (32, [1] * 24, list(range(129, 385, 11))),
         (64, [1] * 24, list(range(129, 385, 11))), (16, [4, 1, 3, 2], [384, 200, 330, 260]), (5, [3, 1], [300, 384])]
CUT = [(16, [1] * 40, list(range(1100, 1900, 20))), (32, [1] * 40, list(range(1100, 1900, 20))),
       (64, [1] * 30, list(range(1300, 1900, 20))), (16, [4, 2, 3] * 8, list(range(700, 1900, 50))), (40, [1, 1], [9000, 700]),
       (128, [1] * 6, list(range(900, 1500, 100)))]
EXPANDED = [(4, [1, 90, 130], [300, 400, 640]), (3, [200, 257], [700, 257 + 400])]
EXPANDED_CUT = [(3, [300, 40], [1900, 2500]), (2, [600], [4100])]


@pytest.mark.gpu
@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("heads,q_lens,seq_lens", WHOLE + CUT)
def test_absorbed(heads, q_lens, seq_lens, latent):
    step = absorbed_step(heads, latent, q_lens, seq_lens, seed=heads + len(q_lens))
    d = step.run()
    torch.cuda.synchronize()
    assert int(d["status"].item()) == 0
    want, mag = step.want()
    check(d["out"], want, mag, BF16, step.logit_size(), latent + 64)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [64, 128])
@pytest.mark.parametrize("heads,q_lens,seq_lens", EXPANDED + EXPANDED_CUT)
def test_expanded(heads, q_lens, seq_lens, size):
    step = expanded_step(heads, size, q_lens, seq_lens, seed=heads + size)
    d = step.run()
    torch.cuda.synchronize()
    assert int(d["status"].item()) == 0
    step.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,q_lens", [(16, [1] * 6), (32, [1] * 6), (64, [1] * 6), (16, [4] * 6)])
@pytest.mark.parametrize("latent", [256, 512])
def test_one_key_of_thousands(heads, q_lens, latent):
    """Logits of thousands that grow from tile to tile, the last key's hundreds above all others': the output is its
    latent, to the roundings of a weight and of the result."""
    n = [70, 130, 384, 900, 2000, 9000][:len(q_lens)]
    step = Step(heads, latent, q_lens, n, BF16, seed=heads, scale=1.0)
    step.q = torch.zeros_like(step.q)
    step.q[..., latent] = 16.0
    for r, s in enumerate(n):
        pos = np.arange(s)
        x = 4.0 * (pos // 64)
        x[s - q_lens[r]] = 4.0 * (s // 64 + 8)  # the first row's own key: the last that every row sees
        step.cache[step.tables[r, pos // 16], pos % 16, latent] = torch.from_numpy(x).to(BF16)
    d = step.run()
    torch.cuda.synchronize()
    assert int(d["status"].item()) == 0
    for r, s in enumerate(n):
        p = s - q_lens[r]
        key = step.cache[step.tables[r, p // 16], p % 16, :latent].double()
        got = d["out"][step.starts[r]:step.starts[r + 1]].double().cpu()
        # (every other weight is below e^-400; the one weight, its sum and the result are off by a rounding each)
        assert ((got - key).abs() <= key.abs() * 2.0 ** -8 * 2).all()


# ---------------------------------------------------------------- the bound is sharp

def online(q, k, v, scale, prior, tile, fault):
    """One head's softmax by tiles in float64, whose references move as the kernels' do; fault(f) is what a move
    multiplies the sums before it by."""
    m = np.full(len(q), -np.inf)
    l, o = np.zeros(len(q)), np.zeros((len(q), v.shape[1]))
    for a in range(0, len(k), tile):
        x = q @ k[a:a + tile].T * scale / np.log(2.0)
        x[np.arange(a, min(a + tile, len(k)))[None] > prior + np.arange(len(q))[:, None]] = -np.inf
        top = x.max(-1)
        up = top > m + 8
        f = np.where(up, np.exp2(m - np.where(up, top, 0.0)), 1.0)
        m = np.where(up, top, m)
        w = np.exp2(x - m[:, None])
        l = l * f + w.sum(-1)
        o = o * (fault(f) if a else f)[:, None] + w @ v[a:a + tile]
    return o / l[:, None]


FAULTS = {"none": lambda f: f, "not applied": np.ones_like, "halved": lambda f: np.where(f < 1, f / 2, f),
          "another row's": lambda f: np.roll(f, 1)}


@pytest.mark.parametrize("latent", [256, 512])
def test_bound_shows_a_wrong_factor(latent):
    heads, q_lens, seq_lens = WHOLE[3]
    step = absorbed_step(heads, latent, q_lens, seq_lens, seed=heads + len(q_lens))
    want, mag = step.want()
    rows = step.cache.double().numpy().reshape(-1, latent + 64)
    for name, fault in FAULTS.items():
        got = np.empty_like(want)
        for r, n in enumerate(step.seq_lens):
            pos = np.arange(n)
            k = rows[step.tables[r, pos // 16] * 16 + pos % 16]
            a, b = step.starts[r], step.starts[r + 1]
            # a tile's rows are (token, head) in turn: all heads of a token share its last key
            for t in range(a, b):
                seen = k[:n - (b - 1 - t)]
                got[t] = online(step.q[t].double().numpy(), seen, seen[:, :latent], step.scale, len(seen), 64, fault)
        over = (np.abs(got - want) > bound(want, mag, BF16, step.logit_size(), latent + 64)).any(-1)
        if name == "none":
            assert not over.any()
        else:
            assert over.mean() > 0.3, (name, over.mean())
