"""Logits of millions over the caches whose softmax weights are held in f16.

A float32 logit of 2^24 (base 2) is known to 2, so the reference that a row's weights are taken from must
not let the largest one leave f16.  With scale 1e6 the logits of N(0, 1) data are N(0, 1.1e7) at
D = 128, and a row is its best key's V where the next best is 1e5 below: float32 sums move a logit by
5e7 x 2^-20 = 50, K rounded to f16 (4-bit chunks) by 1e6 sqrt(128) 2^-11 / sqrt(3) = 3.2e3 rms.
V is rounded to f16 and the result to bf16: 2^-11 x 5 and 2^-8 of it.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import fp8, int4
import paged_kv_attention_04_gb300 as P

from helpers import bits
from test_gpu_int4 import forward, make, spec, wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_attention_04_gb300 import build
    build.build()
    P.lib()


def gaps(cpu, kc):
    """Per row and q head, the best logit less the second best."""
    qsl, out = cpu.query_start_loc.numpy(), np.empty(cpu.q.shape[:2])
    q = wide(cpu.q)
    G = q.shape[1] // kc.shape[2]
    for r, s in enumerate(cpu.spec.seq_lens):
        pos = np.arange(s)
        k = kc[cpu.block_tables.numpy()[r, pos // 16], pos % 16]
        for t in range(qsl[r], qsl[r + 1]):
            n = s - (qsl[r + 1] - 1 - t)
            for h in range(q.shape[1]):
                x = np.sort(k[:n, h // G] @ q[t, h] * cpu.scale)
                out[t, h] = x[-1] - x[-2]
    return out


@pytest.mark.parametrize("kind", ["int4", "fp8"])
@pytest.mark.parametrize("scale", [1e4, 1e6, -1e6])
@pytest.mark.parametrize("q,s", [([1, 1], [3000, 700]), ([5, 15], [2500, 1000]), ([16, 40], [3000, 1000])])
def test_large_logits_pick_the_best_key(q, s, scale, kind):
    cpu, st, kc, vc, lay = make(spec(q, s, seed=190 + q[0]))
    kx, vx = cpu.k_cache.float().numpy(), cpu.v_cache.float().numpy()
    slots = cpu.slot_mapping.numpy()
    kx.reshape(-1, *kx.shape[2:])[slots], vx.reshape(-1, *vx.shape[2:])[slots] = wide(cpu.k), wide(cpu.v)
    if kind == "int4":
        kc, vc = int4.pack(kx, 1.0, False), int4.pack(vx, 1.0, True)
        kd, vd = int4.dequantise(kc, 1.0, False), int4.dequantise(vc, 1.0, True)
    else:
        kc, vc = fp8.encode(kx / 0.0625), fp8.encode(vx / 0.0625)
        lay = P.layout_of(torch.from_numpy(kc), cpu.spec.num_q_heads, k_scale=0.0625, v_scale=0.0625)
        kd, vd = fp8.dequantize(kc, 0.0625), fp8.dequantize(vc, 0.0625)
    cpu.scale = st.scale = scale
    out, flags = forward(st, torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), lay)
    assert flags == 0
    ref = oracle.paged_attention(bits(cpu.q), kd, vd, cpu.block_tables.numpy(), cpu.spec.seq_lens,
                                 cpu.query_start_loc.numpy(), scale, cpu.spec.num_kv_heads)
    got = wide(out)
    assert int((~np.isfinite(got)).sum()) == 0
    clear = gaps(cpu, kd) > 0.1 * abs(scale)
    assert clear.mean() > 0.9
    err = np.abs(got - ref)
    assert int((err > 2.0 ** -11 * 5 + 2.0 ** -8 * np.abs(ref))[clear].sum()) == 0
