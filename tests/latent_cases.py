"""Steps of latent attention for the tests, and the bounds their outputs must keep."""
from __future__ import annotations

import numpy as np
import torch

import paged_kv_attention_04_gb300 as P
from oracle import latent as O


class Step:
    """Requests of q_lens new tokens and seq_lens keys over a latent cache of shuffled blocks, whose slots
    without a token are NaN."""

    def __init__(self, heads, latent, q_lens, seq_lens, dtype=torch.bfloat16, seed=0, offset=0.0, spread=1.0, spare=3,
                 extra_rows=0, scale=None):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.heads, self.latent, self.dtype = heads, latent, dtype
        self.q_lens, self.seq_lens = np.asarray(q_lens, np.int64), np.asarray(seq_lens, np.int64)
        self.starts = np.concatenate([[0], np.cumsum(self.q_lens)])
        nb = -(-self.seq_lens // 16)
        self.blocks = int(nb.sum()) + spare
        perm = rng.permutation(self.blocks)
        self.tables = np.full((len(nb), int(nb.max())), -1, np.int64)
        self.cache = torch.full((self.blocks, 16, latent + 64), float("nan"), dtype=dtype)
        at = 0
        for r, n in enumerate(nb):
            self.tables[r, :n] = perm[at:at + n]
            at += n
            rows = (offset + spread * torch.randn(int(self.seq_lens[r]), latent + 64, generator=g)).to(dtype)
            pos = np.arange(self.seq_lens[r])
            self.cache[self.tables[r, pos // 16], pos % 16] = rows
        self.tokens = int(self.starts[-1])
        self.q = torch.randn(self.tokens + extra_rows, heads, latent + 64, generator=g).to(dtype)[:self.tokens]
        self.scale = scale if scale is not None else 192 ** -0.5

    def gpu(self, device="cuda"):
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(torch.int32).to(device)  # noqa: E731
        return dict(q=self.q.to(device).contiguous(), cache=self.cache.to(device), tables=i32(self.tables),
                    seq=i32(self.seq_lens), qsl=i32(self.starts),
                    out=torch.full((self.tokens, self.heads, self.latent), 7.0, dtype=self.dtype, device=device),
                    status=torch.zeros(1, dtype=torch.int32, device=device))

    def run(self, d=None, max_q=None, max_s=None, layout=None, stream=None):
        d = d or self.gpu()
        lay = layout or P.latent_layout_of(d["cache"], self.heads)
        mq, ms = max_q or int(self.q_lens.max()), max_s or int(self.seq_lens.max())
        if "ws" not in d:
            d["ws"] = P.alloc_latent_workspace(lay, len(d["seq"]), len(d["q"]), mq, ms, device=d["q"].device)
        P.pa_latent_forward(d["q"], d["cache"], d["tables"], d["seq"], d["qsl"], mq, ms, self.scale, d["out"], d["ws"], lay,
                            d["status"], stream)
        return d

    def want(self):
        return O.absorbed(self.q.double().numpy(), self.cache.double().numpy(), self.tables, self.seq_lens, self.starts,
                          self.scale, self.latent)

    def logit_size(self):
        """The largest sum of |q_i k_i| x scale of a query and a key of its request."""
        c = self.cache.double().nan_to_num().abs().flatten(0, 1).numpy()
        big = 0.0
        for r, s in enumerate(self.seq_lens):
            pos = np.arange(s)
            k = c[self.tables[r, pos // 16] * 16 + pos % 16]
            q = self.q[self.starts[r]:self.starts[r + 1]].double().abs().flatten(0, 1).numpy()
            big = max(big, float((q @ k.T).max()))
        return big * abs(self.scale)


def bound(out, mag, dtype, logit_size, width):
    """How far an output may be off: every weight by one rounding to the type (bf16: 2^-8) and by what its
    logit is off, twice for the sum that it is divided by; the result by one rounding more.
    A logit is a float32 sum of `width` products, each partial sum off by at most 2^-23 of the sum
    of magnitudes (the tensor cores truncate), and its scaling and exponential by 2^-21 together;
    float32 sums over the keys add 2^-23 a step, under 2^-12 for the lengths here (4096 steps of a
    tile each at most)."""
    half = torch.finfo(dtype).eps / 2
    logit = logit_size * 1.4427 * width * 2.0 ** -23 + logit_size * 2.0 ** -22
    sums = 2.0 ** -12 if dtype == torch.bfloat16 else 2.0 ** -18
    weight = (half if dtype == torch.bfloat16 else 0.0) + 2 * (logit + 2.0 ** -21) + sums
    return mag * weight + np.abs(out) * half * (1 + 2.0 ** -7) + 1e-30


def check(got, want, mag, dtype, logit_size, width):
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all()
    err, lim = np.abs(g - want), bound(want, mag, dtype, logit_size, width)
    worst = float((err / lim).max())
    assert worst <= 1, f"error {worst:.3g} of its bound, at {np.unravel_index((err / lim).argmax(), err.shape)}"
    return worst
