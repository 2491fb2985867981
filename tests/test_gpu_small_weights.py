"""Softmax weights far below a row's largest over the caches whose weights are held in f16:
4-bit and FP8 (whose K and V values are exact in f16).

Every 32nd key has logit 0 and V = 0 (an attention sink); the others lie `a` nats below, +-0.5,
with V of N(0, 1), so the output is made of the small weights alone and is judged relative to
itself.  Weights are held as f16 of 2^11 P: 11 bits down to 2^-25 of the largest, then steps of
2^-35 of it.

Relative errors of a row of the result, independent from weight to weight and uniform within
their step; w = exp(-a mean(q)) is the row's typical weight, since the keys' mean is -a / sqrt(D)
in every dim and the scale 1 / sqrt(D) (q varies, so w does: mean(q) is 1 +- 0.25 / sqrt(D)):
  output to bf16     2^-8 / sqrt(3) = 2.26e-3
  V values to f16    2^-11 / sqrt(3) = 2.8e-4
  K to f16 (chunks)  |K| < 4: half a step is 2^-10 at most, 2^-10 / sqrt(3) = 5.6e-4 rms a dim; over
                     D dims of q about 1 and a scale of 1 / sqrt(D) a logit is off by that, a
                     weight by as much of itself
  weights            2^-11 / sqrt(3) = 2.8e-4 of each above 2^-25; below it a step is 2^-35, rms
                     2^-35 / sqrt(12), over w
In quadrature, at a = 18 and mean(q) = 1 (w = 2^-26.0), 2.41e-3 in the 2-norm, to which rows of
larger w give the most.  An element is off by half a step, 2^-8 of itself, and five sigma of the
other three, of its row's rms.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import fp8, int4
import paged_kv_attention_04_gb300 as P

from helpers import bits
from test_gpu_int4 import forward, make, reference, spec, wide

pytestmark = pytest.mark.gpu
NORM = 2.5e-3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_attention_04_gb300 import build
    build.build()
    P.lib()


def sinks(cpu, a):
    """K and V pools (float32) as above; q about 1."""
    rng = np.random.default_rng(cpu.spec.seed)
    kc, vc = cpu.k_cache.float().numpy(), cpu.v_cache.float().numpy()
    D = kc.shape[-1]
    bt = cpu.block_tables.numpy()
    for r, s in enumerate(cpu.spec.seq_lens):
        pos = np.arange(s)
        k = rng.standard_normal((s, *kc.shape[2:])) * 0.5 - a / np.sqrt(D)
        v = rng.standard_normal((s, *vc.shape[2:]))
        k[::32], v[::32] = 0, 0
        kc[bt[r, pos // 16], pos % 16], vc[bt[r, pos // 16], pos % 16] = k, v
    q = 1 + 0.25 * rng.standard_normal(cpu.q.shape)
    cpu.q = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16)
    return kc, vc


def close_relative(got, ref, a, q):
    g = wide(got)
    err = np.abs(g - ref)
    rel = np.linalg.norm(err) / np.linalg.norm(ref)
    assert rel <= NORM, f"2-norm {rel:.3g}"
    w = np.exp(-a * wide(q).mean(-1, keepdims=True))
    sigma = np.sqrt(2 * 2.8e-4 ** 2 + 5.6e-4 ** 2 + (2.0 ** -35 / np.sqrt(12) / w) ** 2)
    rms = np.sqrt((ref ** 2).mean(-1, keepdims=True))
    assert (err <= 2.0 ** -8 * np.abs(ref) + 5 * sigma * rms).all()


@pytest.mark.parametrize("a", [14, 18])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,s", [([1, 1], [3000, 700]), ([5, 15], [2500, 1000]), ([16, 40], [3000, 1000])])
def test_small_weights_keep_their_bits(q, s, D, a):
    cpu, st, _, _, lay = make(spec(q, s, D=D, seed=130 + D + a + q[0]))
    kc, vc = sinks(cpu, a)
    kc, vc = int4.pack(kc, 1.0, False), int4.pack(vc, 1.0, True)
    out, flags = forward(st, torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), lay, q=cpu.q.cuda())
    assert flags == 0
    close_relative(out, reference(cpu, kc, vc), a, cpu.q)


@pytest.mark.parametrize("a", [14, 18])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,s", [([1, 1], [3000, 700]), ([5, 15], [2500, 1000]), ([16, 40], [3000, 1000])])
def test_small_weights_keep_their_bits_fp8(q, s, D, a):
    cpu, st, _, _, _ = make(spec(q, s, D=D, seed=150 + D + a + q[0]))
    ks, vs = 0.0625, 0.03125
    kc, vc = (fp8.encode(x / sc) for x, sc in zip(sinks(cpu, a), (ks, vs)))
    lay = P.layout_of(torch.from_numpy(kc), cpu.spec.num_q_heads, k_scale=ks, v_scale=vs)
    out, flags = forward(st, torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), lay, q=cpu.q.cuda())
    assert flags == 0
    ref = oracle.paged_attention(bits(cpu.q), fp8.dequantize(kc, ks), fp8.dequantize(vc, vs), cpu.block_tables.numpy(),
                                 cpu.spec.seq_lens, cpu.query_start_loc.numpy(), cpu.scale, cpu.spec.num_kv_heads)
    close_relative(out, ref, a, cpu.q)
