"""4-bit KV cache: the quantising write stores the oracle's codes and parameters, the
read-back returns the values they stand for, and attention over the cache matches the fp64
oracle over the dequantised cache.

Tolerance of attention against fp64 over the same codes, |v| <= Vmax = 5 times v_scale (N(0, 1)
data).  A rounding is off by at most half a step, relative 2^-8 in bf16 and 2^-11 in f16.
  output          2^-8 |o|
  V values        c s + z to f16: 2^-11 Vmax
  P to f16        2^-11 Vmax (every weight off by 2^-11 of itself)
  logits, chunks  K values to f16, at most 2^-11 of each, uniform: a logit is off by
                  sigma = sqrt(D) / sqrt(D) x 2^-11 / sqrt(3) = 2.8e-4 rms, and moves o by that times
                  sum p |v - o| <= 1; five sigma over the compared outputs
The fixed part is 2^-11 x 10 + 5 x 2.8e-4 = 6.3e-3.  The 2-norm is held too: 2^-8 / sqrt(3) = 2.3e-3
bounds the output's rounding (uniform within half a step), the rest adds under 6e-4 in quadrature
(2^-11 / sqrt(3) twice, and sigma): 2.4e-3 of the result.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import int4
import paged_kv_attention_04_gb300 as P
from paged_kv_attention_04_gb300 import workloads as W

from helpers import bits

pytestmark = pytest.mark.gpu
ATOL, RTOL, NORM = 6.3e-3, 2.0 ** -8, 2.4e-3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_attention_04_gb300 import build
    build.build()
    P.lib()


def wide(t):
    return oracle.widen(bits(t))


def same_cache(got, want, is_v):
    """Codes equal, parameters equal (any NaN is the same as any other)."""
    got = got.cpu().numpy()
    assert np.array_equal(int4.codes(got, is_v), int4.codes(want, is_v))
    for a, b in zip(int4.params(got, is_v), int4.params(want, is_v)):
        assert np.array_equal(a, b, equal_nan=True)


def close(got, ref, vs=1.0):
    g = wide(got)
    assert np.isfinite(g).all()
    err = np.abs(g - ref)
    bad = np.argwhere(~(err <= ATOL * vs + RTOL * np.abs(ref)))
    assert not len(bad), f"{len(bad)} elements off, first {bad[:4].tolist()}, max {err.max():.3g}"
    rel = np.linalg.norm(err) / np.linalg.norm(ref)
    assert rel <= NORM, f"2-norm {rel:.3g}"


def make(spec, ks=1.0, vs=1.0):
    """(cpu step, gpu step, packed K and V pools, layout)."""
    cpu = W.make_step(spec)
    kc0, vc0 = int4.pack(wide(cpu.k_cache), ks, False), int4.pack(wide(cpu.v_cache), vs, True)
    lay = P.layout_of(torch.from_numpy(kc0), spec.num_q_heads, k_scale=ks, v_scale=vs)
    return cpu, cpu.to("cuda"), kc0, vc0, lay


def forward(st, kc, vc, lay, **over):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = P.alloc_workspace(lay, st.spec.num_seqs, st.spec.num_tokens, st.max_seq_len)
    out = torch.full_like(st.q, float("nan"))
    a = dict(bt=st.block_tables, sl=st.seq_lens, q=st.q)
    a.update(over)
    P.pa_forward(a["q"], kc, vc, a["bt"], a["sl"], st.query_start_loc, st.max_query_len, st.max_seq_len,
                 st.scale, out, ws, lay, status)
    torch.cuda.synchronize()
    return out, int(status.item())


def reference(cpu, rk, rv, ks=1.0, vs=1.0):
    return oracle.paged_attention(bits(cpu.q), int4.dequantise(rk, ks, False), int4.dequantise(rv, vs, True),
                                  cpu.block_tables.numpy(), cpu.spec.seq_lens, cpu.query_start_loc.numpy(),
                                  cpu.scale, cpu.spec.num_kv_heads)


def run(spec, ks=1.0, vs=1.0):
    """A whole step: write, attention, the new tokens read back."""
    cpu, st, kc0, vc0, lay = make(spec, ks, vs)
    kc, vc = torch.from_numpy(kc0).cuda(), torch.from_numpy(vc0).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.pa_cache_write(st.k, st.v, st.slot_mapping, kc, vc, lay, status)
    out, flags = forward(st, kc, vc, lay)
    k, v = torch.empty_like(st.k), torch.empty_like(st.v)
    P.pa_cache_read(kc, vc, st.slot_mapping, k, v, lay, status)
    torch.cuda.synchronize()
    assert flags == 0 and int(status.item()) == 0
    rk = int4.store(kc0, wide(cpu.k), cpu.slot_mapping, ks, False)
    rv = int4.store(vc0, wide(cpu.v), cpu.slot_mapping, vs, True)
    same_cache(kc, rk, False)
    same_cache(vc, rv, True)
    slots = cpu.slot_mapping.numpy()
    for got, cache, s, is_v in ((k, rk, ks, False), (v, rv, vs, True)):
        want = int4.dequantise(cache, s, is_v).reshape(-1, *got.shape[1:])[slots]
        assert (np.abs(wide(got) - want) <= np.abs(want) * 2.0 ** -8 + 1e-30).all()
    close(out, reference(cpu, rk, rv, ks, vs), vs)


def spec(q, s, G=4, Hkv=2, D=128, seed=0):
    return W.custom_spec("int4", "bf16", G * Hkv, Hkv, D, q, s, seed=200 + seed)


# ---------------------------------------------------------------- write and read-back

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 3])
@pytest.mark.parametrize("T", [1, 2, 17, 333])
def test_write_and_read(D, Hkv, T):
    """Scattered slots, some skipped, some out of range; untouched slots keep their bytes."""
    rng = np.random.default_rng(T + D + Hkv)
    nb = 40
    x = torch.from_numpy(rng.standard_normal((2, T, Hkv, D)).astype(np.float32)).to(torch.bfloat16)
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    slots[T // 2] = -1 if T > 1 else slots[0]
    device_slots = slots.copy()
    if T > 4:
        slots[1] = -1
        device_slots[1] = nb * 16 + 3
    base = rng.integers(0, 256, (2, nb, Hkv, 10 * D), dtype=np.uint8)
    lay = P.make_layout(4 * Hkv, Hkv, D, nb, torch.bfloat16, cache_dtype=P.PA_INT4, k_scale=0.5, v_scale=3.0)
    kc, vc = (torch.from_numpy(b).cuda() for b in base)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = torch.from_numpy(device_slots).cuda()
    P.pa_cache_write(x[0].cuda(), x[1].cuda(), dev, kc, vc, lay, status)
    torch.cuda.synchronize()
    assert int(status.item()) == (P.PA_DEV_SLOT_RANGE if T > 4 else 0)
    want = [int4.store(base[i], wide(x[i]), slots, s, bool(i)) for i, s in enumerate((0.5, 3.0))]
    assert np.array_equal(kc.cpu().numpy(), want[0]) and np.array_equal(vc.cpu().numpy(), want[1])
    # read back: twice the slots, in reverse, into rows that held something
    status.zero_()
    twice = torch.cat([dev, dev.flip(0)])
    k, v = (torch.full((2 * T, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    P.pa_cache_read(kc, vc, twice, k, v, lay, status)
    torch.cuda.synchronize()
    assert int(status.item()) == (P.PA_DEV_SLOT_RANGE if T > 4 else 0)
    both = np.concatenate([slots, slots[::-1]])
    for got, cache, s, is_v in ((k, want[0], 0.5, False), (v, want[1], 3.0, True)):
        val = int4.dequantise(cache, s, is_v).reshape(nb * 16, Hkv, D)[np.maximum(both, 0)]
        val = np.where((both < 0)[:, None, None], 7.0, val)
        assert (np.abs(wide(got) - val) <= np.abs(val) * 2.0 ** -8 + 1e-30).all()


def test_write_corner_values():
    """Equal values, NaN, infinities, the saturation limit, zeros, tiny and tied values."""
    D, T = 64, 12
    x = np.zeros((T, 2, D), np.float32)
    x[0] = 3.0
    x[1, 0, 5] = np.nan
    x[2, 0, 0], x[2, 0, 1], x[2, 1, 40] = np.inf, -np.inf, np.inf
    x[3] = np.linspace(-1e30, 1e30, 2 * D).reshape(2, D)
    x[4, 0, 0], x[4, 0, 1], x[4, 0, 2] = 30.0, 1.0, 3.0   # s = 2: ties to even
    x[5] = 1e-7 * np.arange(D)                             # f16 subnormal scales
    x[6] = 1e-12 * np.arange(D)                            # scale 0 in f16
    x[7] = -5.0
    x[8] = np.arange(D) - 32.0
    x[9, :, ::2] = 65504.0
    x[10] = 1e-38
    x[11, 1] = np.linspace(-16384, 16384, D)
    xt = torch.from_numpy(x).to(torch.bfloat16)
    lay = P.make_layout(2, 2, D, 2, torch.bfloat16, cache_dtype=P.PA_INT4)
    kc, vc = (torch.zeros(2, 2, 10 * D, dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.arange(T, device="cuda") + 3
    P.pa_cache_write(xt.cuda(), xt.cuda(), slots, kc, vc, lay)
    for cache, is_v in ((kc, False), (vc, True)):
        same_cache(cache, int4.store(np.zeros((2, 2, 10 * D), np.uint8), wide(xt), slots.cpu(), 1.0, is_v), is_v)
    k, v = torch.empty(T, 2, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, 2, D, dtype=torch.bfloat16, device="cuda")
    P.pa_cache_read(kc, vc, slots, k, v, lay)
    assert torch.equal(k.isnan(), v.isnan()) and int(k.isnan().sum()) == 32 and k[1, 0, :32].isnan().all()
    assert torch.equal(k[0], xt[0].cuda()) and torch.equal(v[7], xt[7].cuda())


@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8"])
def test_read_other_caches(kind):
    """A bf16 or fp32 slot comes back bit for bit, an FP8 slot as its value in bf16."""
    nb, Hkv, D = 9, 2, 64
    g = torch.Generator().manual_seed(5)
    if kind == "fp8":
        kc, vc = (torch.randint(0, 256, (nb, 16, Hkv, D), generator=g, dtype=torch.uint8) for _ in range(2))
        lay = P.layout_of(kc, 4, k_scale=0.03, v_scale=1.7)
    else:
        dt = torch.bfloat16 if kind == "bf16" else torch.float32
        kc, vc = (torch.randn(nb, 16, Hkv, D, generator=g).to(dt) for _ in range(2))
        kc[0, 0, 0, 0], vc[1, 2, 1, 3] = float("nan"), float("-inf")
        lay = P.layout_of(kc, 4)
    slots = torch.randint(0, nb * 16, (57,), generator=g)
    slots[3], slots[4] = 0, -1
    out_dt = torch.float32 if kind == "f32" else torch.bfloat16
    k, v = (torch.full((57, Hkv, D), 7.0, dtype=out_dt, device="cuda") for _ in range(2))
    P.pa_cache_read(kc.cuda(), vc.cuda(), slots.cuda(), k, v, lay)
    for got, cache, s in ((k, kc, 0.03), (v, vc, 1.7)):
        rows = cache.view(nb * 16, Hkv, D)[slots.clamp(min=0)]
        if kind == "fp8":
            rows = (rows.view(torch.float8_e4m3fn).float() * torch.tensor(s)).to(torch.bfloat16)
        rows[4] = 7.0
        assert torch.equal(got.cpu().nan_to_num(9e9), rows.nan_to_num(9e9))


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_decode(D, G):
    """One token to several splits, lengths at and around block ends."""
    run(spec([1] * 9, [1, 2, 15, 16, 17, 64, 700, 2049, 5000], G=G, D=D, seed=D + G), 0.5, 2.0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_few_tokens(D, G):
    """2 to 15 new tokens: the causal edge inside and across blocks and tiles."""
    run(spec([2, 15, 7, 3, 1, 9, 2], [2, 15, 40, 18, 33, 2100, 4100], G=G, D=D, seed=10 + D + G), 2.0, 0.5)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_chunks(D, G):
    """Chunks from 16 tokens on, alone and after a prior context."""
    run(spec([16, 17, 130, 1, 40], [16, 300, 130, 77, 1501], G=G, D=D, seed=20 + D + G))


def test_chunk_pieces():
    """A short chunk after a long prior: the KV cut into pieces that are merged."""
    run(spec([16, 1], [6016, 300], seed=31), 0.25, 4.0)


def test_many_requests():
    """More requests than the plan's CTA has threads, one block each, then long ones."""
    run(spec([1] * 300 + [5, 20], list(range(1, 301)) + [2000, 2500], D=64, seed=32))


def test_mixed_step():
    s = W.spec_mixed_step()
    run(W.custom_spec("int4-mixed", "bf16", 32, 8, 128, np.concatenate([s.q_lens[:40], s.q_lens[-2:]]),
                      np.concatenate([s.seq_lens[:40], s.seq_lens[-2:]]), shared_prefix_blocks=64,
                      sharing=np.concatenate([s.sharing[:40], [False, False]]), seed=33))


def test_unwritten_slots_and_other_blocks_do_not_matter():
    """The pool's unwritten slots have NaN parameters (make_step's NaN); with any other
    bytes there the result is the same to the bit."""
    for q, s in (([1, 1], [5, 300]), ([3, 9], [20, 333]), ([20, 33], [20, 300])):
        cpu, st, kc0, vc0, lay = make(spec(q, s, seed=40 + q[0]))
        kc0 = int4.store(kc0, wide(cpu.k), cpu.slot_mapping, 1.0, False)
        vc0 = int4.store(vc0, wide(cpu.v), cpu.slot_mapping, 1.0, True)
        a, fa = forward(st, torch.from_numpy(kc0).cuda(), torch.from_numpy(vc0).cuda(), lay)
        zero_k, zero_v = kc0.copy(), vc0.copy()
        for cache, is_v in ((zero_k, False), (zero_v, True)):
            sc, _ = int4.params(cache, is_v)
            empty = np.nonzero(np.isnan(sc[:, :, 0, 0]).ravel())[0]
            assert len(empty)
            rows = np.random.default_rng(1).standard_normal((len(empty), *cpu.k.shape[1:])) * 50
            cache[:] = int4.store(cache, rows, empty, 1.0, is_v)
        b, fb = forward(st, torch.from_numpy(zero_k).cuda(), torch.from_numpy(zero_v).cuda(), lay)
        assert fa == 0 and fb == 0
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("q,s", [([1], [40]), ([5], [40]), ([20], [40])])
def test_bad_block_ids_are_flagged_and_read_as_zeros(q, s):
    cpu, st, kc0, vc0, lay = make(spec(q, s, seed=50))
    kc0 = int4.store(kc0, wide(cpu.k), cpu.slot_mapping, 1.0, False)
    vc0 = int4.store(vc0, wide(cpu.v), cpu.slot_mapping, 1.0, True)
    bad = cpu.block_tables[0, 1].item()
    for wrong in (lay.num_blocks + 5, -7, 1 << 30, -1):
        bt = st.block_tables.clone()
        bt[0, 1] = wrong
        out, flags = forward(st, torch.from_numpy(kc0).cuda(), torch.from_numpy(vc0).cuda(), lay, bt=bt)
        assert flags == P.PA_DEV_BLOCK_RANGE
        zk, zv = kc0.copy(), vc0.copy()
        zk[bad], zv[bad] = 0, 0
        close(out, reference(cpu, zk, zv))


@pytest.mark.parametrize("amp", [1e-30, 1e-6, 300.0, 1e30])
def test_query_range_of_short_queries(amp):
    """Short queries scale q by a power of two, so its magnitude is free: logits are as
    large as before when the softmax scale is divided by it."""
    cpu, st, kc0, vc0, lay = make(spec([1, 4], [333, 200], seed=60))
    kc0 = int4.store(kc0, wide(cpu.k), cpu.slot_mapping, 1.0, False)
    vc0 = int4.store(vc0, wide(cpu.v), cpu.slot_mapping, 1.0, True)
    cpu.q = (cpu.q.float() * amp).to(torch.bfloat16)
    st.q = cpu.q.cuda()
    cpu.scale = st.scale = st.scale / amp
    out, flags = forward(st, torch.from_numpy(kc0).cuda(), torch.from_numpy(vc0).cuda(), lay)
    assert flags == 0
    close(out, reference(cpu, kc0, vc0))


def test_large_logits_and_late_maxima():
    """Logits of several hundred that grow along the keys: the running maximum moves block
    after block; and a query of zeros weighs all keys alike."""
    for q, s in (([1, 1], [700, 2500]), ([6, 3], [700, 2500]), ([33, 16], [700, 2500])):
        cpu, st, kc0, vc0, lay = make(spec(q, s, seed=70 + q[0]))
        cpu.q[0] = 0
        ramp = torch.arange(max(s)) / max(s) * 6
        kc = cpu.k_cache.float()
        for r in range(len(s)):
            pos = torch.arange(s[r])
            kc[cpu.block_tables[r, pos // 16].long(), pos % 16] *= ramp[pos][:, None, None] + 0.1
        kc0 = int4.pack(kc.numpy(), 1.0, False)
        kc0 = int4.store(kc0, wide(cpu.k), cpu.slot_mapping, 1.0, False)
        vc0 = int4.store(vc0, wide(cpu.v), cpu.slot_mapping, 1.0, True)
        st.q = cpu.q.cuda()
        cpu.scale = st.scale = 0.5
        if q[0] >= 16:   # chunks round K to f16 first: keep its error in the logits small
            cpu.scale = st.scale = 0.02
        out, flags = forward(st, torch.from_numpy(kc0).cuda(), torch.from_numpy(vc0).cuda(), lay)
        assert flags == 0
        close(out, reference(cpu, kc0, vc0))


def test_nan_value_reaches_only_its_request():
    cpu, st, kc0, vc0, lay = make(spec([1, 4, 20], [40, 41, 42], seed=80))
    kc0 = int4.store(kc0, wide(cpu.k), cpu.slot_mapping, 1.0, False)
    vc0 = int4.store(vc0, wide(cpu.v), cpu.slot_mapping, 1.0, True)
    x = wide(cpu.v)[:1].copy()
    x[:, 0, 3] = np.nan   # kv head 0, first group, of request 1's position 7
    slot = int(cpu.block_tables[1, 0]) * 16 + 7
    vc0 = int4.store(vc0, x, [slot], 1.0, True)
    out, flags = forward(st, torch.from_numpy(kc0).cuda(), torch.from_numpy(vc0).cuda(), lay)
    nan = out.isnan().cpu()
    assert flags == 0 and nan[1:5, :4, :32].all()
    nan[1:5, :4, :32] = False
    assert not nan.any()


def test_noalloc_and_serial_schedule_give_the_same_bits():
    cpu, st, kc0, vc0, lay = make(spec([1, 1, 5, 64], [700, 20, 90, 300], seed=90))
    kc, vc = torch.from_numpy(kc0).cuda(), torch.from_numpy(vc0).cuda()
    P.pa_cache_write(st.k, st.v, st.slot_mapping, kc, vc, lay)
    a, _ = forward(st, kc, vc, lay)
    b = torch.empty_like(a)
    P.pa_forward_noalloc(st.q, kc, vc, st.block_tables, st.seq_lens, st.query_start_loc, st.max_query_len,
                         st.max_seq_len, st.scale, b, lay)
    P.pa_set_prefill_overlap(False)
    try:
        c, _ = forward(st, kc, vc, lay)
    finally:
        P.pa_set_prefill_overlap(True)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.equal(a.view(torch.int16), c.view(torch.int16))


def test_captured_step_replays_with_new_inputs():
    """Write, attention and read-back on a side stream, captured and replayed; a second
    graph with its own workspace runs between the replays."""
    graphs = []
    for seed in (95, 96):
        cpu, st, kc0, vc0, lay = make(spec([1, 1, 3, 40], [700, 20, 90, 300], seed=seed))
        kc, vc = torch.from_numpy(kc0).cuda(), torch.from_numpy(vc0).cuda()
        ws = P.alloc_workspace(lay, 4, st.spec.num_tokens, st.max_seq_len)
        out, k, v = torch.empty_like(st.q), torch.empty_like(st.k), torch.empty_like(st.v)

        def step(st=st, kc=kc, vc=vc, ws=ws, out=out, k=k, v=v, lay=lay):
            P.pa_cache_write(st.k, st.v, st.slot_mapping, kc, vc, lay)
            P.pa_forward(st.q, kc, vc, st.block_tables, st.seq_lens, st.query_start_loc, st.max_query_len,
                         st.max_seq_len, st.scale, out, ws, lay)
            P.pa_cache_read(kc, vc, st.slot_mapping, k, v, lay)
        step()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        graphs.append((g, st, out, k, v, step))
    for turn in range(2):
        for g, st, out, k, v, step in graphs:
            for x in (st.q, st.k, st.v):
                x.copy_(torch.randn_like(x.float()).to(x.dtype))
            g.replay()
            torch.cuda.synchronize()
            got = [x.clone() for x in (out, k, v)]
            step()
            torch.cuda.synchronize()
            for a, b in zip(got, (out, k, v)):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-30])
def test_softmax_scale_zero_negative_tiny(scale):
    """The sign of the scale is folded into the staged q; a scale of zero weighs all visible
    keys alike."""
    cpu, st, kc0, vc0, lay = make(spec([1, 1, 5, 3, 20], [33, 700, 300, 40, 130], seed=100))
    kc0 = int4.store(kc0, wide(cpu.k), cpu.slot_mapping, 1.0, False)
    vc0 = int4.store(vc0, wide(cpu.v), cpu.slot_mapping, 1.0, True)
    cpu.scale = st.scale = scale
    out, flags = forward(st, torch.from_numpy(kc0).cuda(), torch.from_numpy(vc0).cuda(), lay)
    assert flags == 0
    close(out, reference(cpu, kc0, vc0))


@pytest.mark.parametrize("D,G,Hkv,q,s", [
    (64, 8, 1, [1, 1], [40000, 9]),         # 20 and more splits of one tile, merged by a CTA
    (128, 1, 3, [1, 4, 17], [9000, 5000, 4000]),
    (64, 2, 5, [1, 15, 33], [300, 4100, 2100]),
])
def test_long_and_odd_heads(D, G, Hkv, q, s):
    run(spec(q, s, G=G, Hkv=Hkv, D=D, seed=110 + D + Hkv))


def test_two_steps_on_two_streams():
    """Two steps with their own workspaces, one on each of two streams at once, give the bits
    that they give alone."""
    steps = []
    for seed in (120, 121):
        cpu, st, kc0, vc0, lay = make(spec([1] * 20 + [3, 7], [900] * 20 + [800, 500], seed=seed))
        kc, vc = torch.from_numpy(kc0).cuda(), torch.from_numpy(vc0).cuda()
        P.pa_cache_write(st.k, st.v, st.slot_mapping, kc, vc, lay)
        alone, _ = forward(st, kc, vc, lay)
        ws = P.alloc_workspace(lay, st.spec.num_seqs, st.spec.num_tokens, st.max_seq_len)
        steps.append((st, kc, vc, lay, ws, torch.empty_like(alone), alone, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for st, kc, vc, lay, ws, out, alone, stream in steps:
            P.pa_forward(st.q, kc, vc, st.block_tables, st.seq_lens, st.query_start_loc, st.max_query_len,
                         st.max_seq_len, st.scale, out, ws, lay, stream=stream)
    torch.cuda.synchronize()
    for st, kc, vc, lay, ws, out, alone, stream in steps:
        assert torch.equal(out.view(torch.int16), alone.view(torch.int16))


def test_binding_refuses_what_would_run_out_of_bounds():
    kc = torch.zeros(4, 2, 640, dtype=torch.uint8, device="cuda")
    lay = P.layout_of(kc, 8)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(P.PaError, match="rows"):
        P.pa_cache_read(kc, kc, slots, k[:2].contiguous(), k, lay)
    with pytest.raises(P.PaError, match="rows"):
        P.pa_cache_read(kc, kc, slots, k, k.float(), lay)
    with pytest.raises(P.PaError, match="slot_mapping"):
        P.pa_cache_read(kc, kc, slots.int(), k, k.clone(), lay)
    with pytest.raises(P.PaError, match="slots for"):
        P.pa_cache_write(k, k, slots[:2].contiguous(), kc, kc.clone(), lay)
    for wrong in (kc[:3].contiguous(), torch.zeros(4, 16, 2, 64, dtype=torch.uint8, device="cuda"), kc.to(torch.int32)):
        for call in (lambda: P.pa_cache_write(k, k, slots, wrong, kc, lay),
                     lambda: P.pa_cache_read(kc, wrong, slots, k, k.clone(), lay)):
            with pytest.raises(P.PaError, match="4-bit cache"):
                call()
    with pytest.raises(P.PaError, match="not contiguous"):
        P.pa_cache_read(kc, kc, slots, k.transpose(1, 2), k, lay)
