"""The rotating slot write: bits against the formula in float32 and against rotating first and
writing then, errors against 64 bits, slices, skipped tokens and bad inputs."""
import numpy as np
import pytest
import torch

import paged_kv_attention_04_gb300 as P
from oracle import latent as O

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_attention_04_gb300 import build
    build.build()
    P.lib()


def rotated(x, tab, pos, pairs):
    """The formula in float32, products rounded one by one, then rounded to x's type (CPU)."""
    n = tab.shape[1]
    row = tab[pos][:, None]
    c, s = row[..., :n // 2], row[..., n // 2:]
    y = x.float().clone()
    ia, ib = (slice(0, n, 2), slice(1, n, 2)) if pairs else (slice(0, n // 2), slice(n // 2, n))
    a, b = y[..., ia].clone(), y[..., ib].clone()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y.to(x.dtype)


def case(tokens, hq, hkv, d, n, dtype=BF16, cache=None, seed=0, scales=(1.0, 1.0)):
    g = torch.Generator().manual_seed(seed)
    blocks = tokens // 16 + 3
    lay = P.make_layout(hq, hkv, d, blocks, dtype, cache_dtype=cache, k_scale=scales[0], v_scale=scales[1])
    qkv = torch.randn(tokens, (hq + 2 * hkv) * d, generator=g).to(dtype)
    q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], -1))
    pos = torch.randint(0, 500, (tokens,), generator=g)
    tab = torch.from_numpy(O.table(500, n)).float()
    slots = torch.randperm(blocks * 16, generator=g)[:tokens]
    shape = P.cache_shape(lay)
    if cache is None:
        kc, vc = torch.randn(2, *shape, generator=g).to(dtype)
    else:
        kc, vc = torch.randint(0, 256, (2, *shape), generator=g, dtype=torch.uint8)
    return lay, qkv, q, k, v, pos, tab, slots, kc, vc


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu()


def on_gpu(qkv, hq, hkv, d):
    """The slices of the projection, on the GPU."""
    x = qkv.cuda()
    return [y.unflatten(-1, (-1, d)) for y in x.split([hq * d, hkv * d, hkv * d], -1)]


CACHES = [(BF16, None), (F32, None), (BF16, P.PA_FP8_E4M3), (BF16, P.PA_INT4)]


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("tokens,hq,hkv,d,n", [(1, 1, 1, 64, 64), (5, 4, 2, 64, 48), (37, 8, 8, 128, 128),
                                               (130, 32, 4, 128, 64), (3, 8, 1, 128, 16), (16, 2, 1, 64, 32)])
def test_bits(tokens, hq, hkv, d, n, dtype, cache, pairs):
    scales = (0.37, 1.7) if cache else (1.0, 1.0)
    lay, qkv, q, k, v, pos, tab, slots, kc, vc = case(tokens, hq, hkv, d, n, dtype, cache, tokens + n, scales)
    gq, gk, gv = on_gpu(qkv, hq, hkv, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.zeros(tokens, hq, d, dtype=dtype, device="cuda")
    got = kc.cuda(), vc.cuda()
    P.pa_rope_cache_write(gq, gk, gv, pos.cuda(), tab.cuda(), slots.cuda(), q_out, *got, lay, pairs=pairs, status=status)
    # the keys rotated first, written then
    kr = rotated(k, tab, pos, pairs)
    want = kc.cuda(), vc.cuda()
    P.pa_cache_write(kr.cuda(), v.contiguous().cuda(), slots.cuda(), *want, lay, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(bits(q_out), bits(rotated(q, tab, pos, pairs)))
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))
    # against 64 bits: two products and a sum in float32, one rounding to the type
    exact = O.rotate(q.double().numpy(), tab.double().numpy(), pos.numpy(), pairs)
    big = np.abs(q.double().numpy()).max(-1, keepdims=True)
    eps = 0.0 if dtype == F32 else torch.finfo(dtype).eps / 2
    assert (np.abs(q_out.double().cpu().numpy() - exact) <= eps * np.abs(exact) * (1 + 2 ** -7) + 4 * 2.0 ** -24 * 2 * big).all()


@pytest.mark.parametrize("tokens,hq,hkv,d,cache", [(60000, 3, 3, 64, None), (45000, 4, 1, 128, None), (30000, 3, 3, 128, None),
                                                   (33000, 8, 1, 128, P.PA_INT4)])
def test_many_tokens(tokens, hq, hkv, d, cache):
    """Steps whose rows are taken two at a time (odd numbers of them too), with skipped tokens: as in parts."""
    lay, qkv, q, k, v, pos, tab, slots, kc, vc = case(tokens, hq, hkv, d, 32, BF16, cache, seed=7)
    slots[::97] = -1
    gq, gk, gv = on_gpu(qkv, hq, hkv, d)
    gpos, gtab, gslots = pos.cuda(), tab.cuda(), slots.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    whole, parts = (kc.cuda(), vc.cuda()), (kc.cuda(), vc.cuda())
    q_out, q_parts = (torch.zeros(tokens, hq, d, dtype=BF16, device="cuda") for _ in range(2))
    P.pa_rope_cache_write(gq, gk, gv, gpos, gtab, gslots, q_out, *whole, lay, status=status)
    for i in range(0, tokens, 5000):
        at = slice(i, i + 5000)
        P.pa_rope_cache_write(gq[at], gk[at], gv[at], gpos[at], gtab, gslots[at], q_parts[at], *parts, lay, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(bits(q_out), bits(q_parts))
    assert torch.equal(bits(q_out[-3000:]), bits(rotated(q[-3000:], tab, pos[-3000:], False)))
    for a, b in zip(whole, parts):
        assert torch.equal(bits(a), bits(b))


def test_in_place_and_keys_alone():
    lay, qkv, q, k, v, pos, tab, slots, kc, vc = case(33, 8, 2, 128, 128, seed=5)
    gq = q.contiguous().cuda()
    got = kc.cuda(), vc.cuda()
    args = pos.cuda(), tab.cuda(), slots.cuda()
    P.pa_rope_cache_write(gq, k.contiguous().cuda(), v.contiguous().cuda(), *args, gq, *got, lay)
    alone = kc.cuda(), vc.cuda()
    P.pa_rope_cache_write(None, k.contiguous().cuda(), v.contiguous().cuda(), *args, None, *alone, lay)
    torch.cuda.synchronize()
    assert torch.equal(bits(gq), bits(rotated(q, tab, pos, False)))
    for a, b in zip(got, alone):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("dtype,cache", CACHES)
def test_skipped_and_bad_tokens(dtype, cache):
    """A negative slot skips the write, not q; a slot or position out of range is skipped and flagged;
    the others are written."""
    lay, qkv, q, k, v, pos, tab, slots, kc, vc = case(9, 4, 2, 64, 64, dtype, cache, seed=2)
    slots[1], slots[3] = -1, lay.num_blocks * 16
    pos[5], pos[7] = -1, 500
    q_out = torch.full((9, 4, 64), 7.0, dtype=dtype, device="cuda")
    got = kc.cuda(), vc.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.pa_rope_cache_write(*on_gpu(qkv, 4, 2, 64), pos.cuda(), tab.cuda(), slots.cuda(), q_out, *got, lay, status=status)
    keep = torch.tensor([0, 2, 4, 6, 8])
    want = kc.cuda(), vc.cuda()
    P.pa_cache_write(rotated(k[keep], tab, pos[keep], False).cuda(), v[keep].contiguous().cuda(), slots[keep].cuda(), *want, lay)
    torch.cuda.synchronize()
    assert int(status.item()) == P.PA_DEV_SLOT_RANGE | P.PA_DEV_POSITION
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))
    turned = [0, 1, 2, 3, 4, 6, 8]
    assert torch.equal(bits(q_out[turned]), bits(rotated(q[turned], tab, pos[turned], False)))
    assert (q_out[[5, 7]] == 7).all()


def test_captured_and_replayed():
    """A graph rotates what its inputs hold at replay."""
    lay, qkv, q, k, v, pos, tab, slots, kc, vc = case(20, 8, 2, 128, 128, seed=9)
    gq, gk, gv = on_gpu(qkv, 8, 2, 128)
    got, tab_g, slots_g, pos_g = (kc.cuda(), vc.cuda()), tab.cuda(), slots.cuda(), pos.cuda()
    q_out = torch.zeros(20, 8, 128, dtype=BF16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.pa_rope_cache_write(gq, gk, gv, pos_g, tab_g, slots_g, q_out, *got, lay)
    new = (pos + 3) % 500
    pos_g.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(q_out), bits(rotated(q, tab, new, False)))
    assert torch.equal(bits(got[0].flatten(0, 1)[slots_g]), bits(rotated(k, tab, new, False)))
