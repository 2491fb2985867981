"""Edges of the 4-bit cache: bad block-table entries in later tiles of a chunk, K values far from
zero, pages issued across many short units.  Tolerances as in test_gpu_int4.py unless derived at
the test."""
import numpy as np
import pytest
import torch

from oracle import int4
import paged_kv_attention_04_gb300 as P

from test_gpu_int4 import close, forward, make, reference, spec, wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_attention_04_gb300 import build
    build.build()
    P.lib()


def filled(sp):
    """A step whose new tokens are in the pools: (cpu step, gpu step, K pool, V pool, layout)."""
    cpu, st, kc, vc, lay = make(sp)
    kc = int4.store(kc, wide(cpu.k), cpu.slot_mapping, 1.0, False)
    vc = int4.store(vc, wide(cpu.v), cpu.slot_mapping, 1.0, True)
    return cpu, st, kc, vc, lay


@pytest.mark.parametrize("q", [16, 300])
def test_bad_block_ids_in_later_tiles_read_as_zeros(q):
    """Several per 128-key tile, in tiles whose staging buffer held another tile's pages."""
    cpu, st, kc, vc, lay = filled(spec([q], [1700], seed=160 + q))
    bt = st.block_tables.clone()
    zk, zv = kc.copy(), vc.copy()
    for i, b in enumerate((1, 17, 18, 23, 40, 41, 42, 43, 44, 45, 46, 47, 70, 105)):
        zk[cpu.block_tables[0, b]] = zv[cpu.block_tables[0, b]] = 0
        bt[0, b] = (-1, lay.num_blocks, 1 << 30)[i % 3]
    out, flags = forward(st, torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), lay, bt=bt)
    assert flags == P.PA_DEV_BLOCK_RANGE
    close(out, reference(cpu, zk, zv))


@pytest.mark.parametrize("q", [1, 3])
def test_units_shorter_than_the_ring(q):
    """Requests of one to four blocks and a few longer ones: a warp's stream runs on into units
    that are published while it asks for them; the results repeat to the bit."""
    lens = [(7 * i) % 61 + q for i in range(700)] + [900, 2000]
    cpu, st, kc, vc, lay = filled(spec([q] * len(lens), lens, D=64, seed=170 + q))
    kc, vc = torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda()
    a, flags = forward(st, kc, vc, lay)
    assert flags == 0
    close(a, reference(cpu, kc.cpu().numpy(), vc.cpu().numpy()))
    for _ in range(10):
        b, _ = forward(st, kc, vc, lay)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,s", [([1, 1], [2500, 300]), ([7, 15], [2500, 300]), ([40, 130], [2500, 300])])
def test_keys_far_from_zero(q, s, D):
    """K of 30 + N(0, 1): a group's zero is 90 of its steps.

    Queries below 16 tokens use K as the codes say (z against the group sums of q, kept to 2^-15 of
    the row's largest q; z differs by 0.4 between keys: under 1e-5 in a logit): tolerances unchanged.
    Chunks round K to f16: half a step is 2^-7 below 32, 2^-6 above (2.3 % of the values), 4.7e-3 rms;
    over D dims of q of N(0, 1) and a scale of 1 / sqrt(D) a logit is off by as much, and o by
    that times |v - o|: sqrt(4.7e-3^2 + 2.4e-3^2) = 5.3e-3 in the 2-norm, an element by the
    2^-11 x 10 and 2^-8 |o| of the other roundings and five sigma, 2.84e-2."""
    cpu, st, kc, vc, lay = filled(spec(q, s, D=D, seed=180 + D + q[0]))
    pool = 30 + cpu.k_cache.float().numpy()
    bt = cpu.block_tables.numpy()
    for r, n in enumerate(s):   # this step's tokens too
        pos = np.arange(n - q[r], n)
        pool[bt[r, pos // 16], pos % 16] = 30 + wide(cpu.k)[cpu.query_start_loc[r]:cpu.query_start_loc[r + 1]]
    kc = int4.pack(pool, 1.0, False)
    out, flags = forward(st, torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), lay)
    assert flags == 0
    ref = reference(cpu, kc, vc)
    if q[0] < 16:
        close(out, ref)
        return
    err = np.abs(wide(out) - ref)
    assert (err <= 2.84e-2 + 2.0 ** -8 * np.abs(ref)).all()
    assert np.linalg.norm(err) <= 5.3e-3 * np.linalg.norm(ref)


@pytest.mark.parametrize("q,s", [([1, 1], [700, 40]), ([5, 3], [700, 40]), ([16, 20], [700, 40])])
def test_a_k_scale_beyond_the_data_gives_keys_of_zero(q, s):
    """K of N(0, 1) over a scale of 1e37 has codes, scales and zeros of 0: all keys weigh alike.
    The scale itself times the largest q is past float32."""
    cpu, st, _, vc, lay = filled(spec(q, s, seed=200 + q[0]))
    x = cpu.k_cache.float().numpy()
    x.reshape(-1, *x.shape[2:])[cpu.slot_mapping.numpy()] = wide(cpu.k)
    kc = int4.pack(x, 1e37, False)
    lay.k_scale = 1e37
    out, flags = forward(st, torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), lay)
    assert flags == 0
    close(out, reference(cpu, kc, vc, ks=1e37))


def test_pages_past_4_gib_and_off_alignment():
    """Blocks whose pages lie more than 2^32 bytes into the cache, in caches that start 16 bytes off a
    larger alignment: write, every attention path and read-back give what a small pool gives."""
    cpu, st, kc, vc, lay = make(spec([1, 1, 5, 40], [700, 20, 90, 300], Hkv=8, seed=210))
    nb = lay.num_blocks
    big = (1 << 32) // (8 * 1280) + 2 * nb
    ids = torch.randperm(nb) + big - nb   # block i of the small pool is block ids[i] of the large one

    def step(kc, vc, lay, bt, slots):
        P.pa_cache_write(st.k, st.v, slots, kc, vc, lay)
        out, flags = forward(st, kc, vc, lay, bt=bt)
        k, v = torch.empty_like(st.k), torch.empty_like(st.v)
        P.pa_cache_read(kc, vc, slots, k, v, lay)
        assert flags == 0
        return out, k, v

    want = step(torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), lay, st.block_tables, st.slot_mapping)
    large = [torch.empty(16 + big * 8 * 1280, dtype=torch.uint8, device="cuda")[16:].view(big, 8, 1280) for _ in range(2)]
    for c, small in zip(large, (kc, vc)):
        c[ids.cuda()] = torch.from_numpy(small).cuda()
    bt, slots = cpu.block_tables.long(), cpu.slot_mapping
    bt = torch.where(bt < 0, bt, ids[bt.clamp(min=0)]).int().cuda()
    got = step(*large, P.layout_of(large[0], st.spec.num_q_heads), bt, (ids[slots // 16] * 16 + slots % 16).cuda())
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
