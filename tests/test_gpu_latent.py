"""The latent cache: write, read-back and absorbed attention."""
import numpy as np
import pytest
import torch

import paged_kv_attention_04_gb300 as P
from latent_cases import Step, check
from oracle import latent as O

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_attention_04_gb300 import build
    build.build()
    P.lib()


# ---------------------------------------------------------------- write and read-back

def write_case(tokens, heads, latent, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    blocks = tokens // 16 + 2
    row = torch.randn(tokens, latent + 64 + 8, generator=g).to(dtype)  # a projection's rows
    q = torch.randn(tokens, heads, 128 + 64, generator=g).to(dtype)
    pos = torch.randint(0, 300, (tokens,), generator=g)
    tab = torch.from_numpy(O.table(300, 64)).float()
    slots = torch.randperm(blocks * 16, generator=g)[:tokens]
    cache = torch.randn(blocks, 16, latent + 64, generator=g).to(dtype)
    weight = (1 + 0.2 * torch.randn(latent, generator=g)).to(dtype)
    return row, q, pos, tab, slots, cache, weight


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,heads,latent", [(1, 1, 256), (7, 20, 512), (33, 128, 256), (65, 8, 512), (2, 9, 512)])
def test_write_and_read(tokens, heads, latent, dtype, norm, pairs):
    row, q, pos, tab, slots, cache, weight = write_case(tokens, heads, latent, dtype, tokens + heads)
    lay = P.make_latent_layout(heads, latent, cache.shape[0], dtype)
    grow, gq, gc = row.cuda(), q.cuda(), cache.cuda()
    q_abs = torch.full((tokens, heads, latent + 64), 7.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.pa_latent_write(grow[:, :latent], grow[:, latent:latent + 64], gq[..., 128:], pos.cuda(), tab.cuda(), slots.cuda(),
                      q_abs[..., latent:], gc, lay, norm_weight=weight.cuda() if norm else None, eps=1e-5, pairs=pairs,
                      status=status)
    c_out, k_out = torch.empty(tokens, latent, dtype=dtype, device="cuda"), torch.empty(tokens, 64, dtype=dtype, device="cuda")
    P.pa_latent_read(gc, slots.cuda(), c_out, k_out, lay, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert (q_abs[..., :latent] == 7).all()
    tab64 = tab.double().numpy()
    half = torch.finfo(dtype).eps / 2
    f32 = 2.0 ** -24
    for got, x in ((q_abs[..., latent:], q[..., 128:]), (k_out, row[:, latent:latent + 64])):
        x = x.double().numpy()
        want = O.rotate(x, tab64, pos.numpy(), pairs)
        # two products and their sum, each rounded; then one rounding to the type
        lim = half * np.abs(want) * (1 + 2 ** -7) + 4 * f32 * 2 * np.abs(x).max(-1, keepdims=True)
        assert (np.abs(got.double().cpu().numpy() - want) <= lim).all()
    c = row[:, :latent]
    if norm:
        want = O.rms_norm(c.double().numpy(), weight.double().numpy(), 1e-5)
        # a sum of R squares (R / 32 + 5 roundings a lane, halved by the root), root, division, two products
        lim = np.abs(want) * (half * (1 + 2 ** -7) + f32 * (latent / 64 + 3 + 6))
        assert (np.abs(c_out.double().cpu().numpy() - want) <= lim).all()
    else:
        assert torch.equal(c_out.cpu(), c)
    # the row is what the read-back gave, and no other slot changed
    want = cache.flatten(0, 1).clone()
    want[slots] = torch.cat([c_out, k_out], -1).cpu()
    assert torch.equal(gc.flatten(0, 1).cpu(), want)


def test_write_skips_and_flags():
    row, q, pos, tab, slots, cache, weight = write_case(9, 4, 512, BF16, 3)
    slots[1], slots[3] = -1, cache.shape[0] * 16 + 5
    pos[5], pos[7] = -1, 300
    lay = P.make_latent_layout(4, 512, cache.shape[0])
    gc = cache.cuda()
    q_out = torch.full((9, 4, 64), 7.0, dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = row.cuda()
    P.pa_latent_write(g[:, :512], g[:, 512:576], q.cuda()[..., 128:], pos.cuda(), tab.cuda(), slots.cuda(), q_out, gc, lay,
                      status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == P.PA_DEV_SLOT_RANGE | P.PA_DEV_POSITION
    keep = [0, 2, 4, 6, 8]
    want = cache.flatten(0, 1).clone()
    turned = O.rotate(row[:, 512:576].double().numpy(), tab.double().numpy(), pos.clamp(0, 299).numpy(), False)
    got = gc.flatten(0, 1).cpu()
    assert torch.equal(got[slots[keep]][:, :512], row[keep, :512])
    assert np.abs(got[slots[keep]][:, 512:].double().numpy() - turned[keep]).max() < 0.05
    untouched = torch.ones(len(want), dtype=torch.bool)
    untouched[slots[keep]] = False
    assert torch.equal(got[untouched], want[untouched])
    assert (q_out[[5, 7]] == 7).all() and (q_out[[0, 1, 2, 3, 4, 6, 8]] != 7).any(-1).all()
    # read-back: skipped rows stay, slots may repeat
    c_out, k_out = torch.full((9, 512), 7.0, dtype=BF16, device="cuda"), torch.full((9, 64), 7.0, dtype=BF16, device="cuda")
    status.zero_()
    slots[8] = slots[0]
    P.pa_latent_read(gc, slots.cuda(), c_out, k_out, lay, status)
    torch.cuda.synchronize()
    assert int(status.item()) == P.PA_DEV_SLOT_RANGE
    assert (c_out[[1, 3]] == 7).all() and (k_out[[1, 3]] == 7).all()
    assert torch.equal(c_out[8], c_out[0]) and torch.equal(torch.cat([c_out, k_out], -1)[0].cpu(), got[slots[0]])


def test_write_in_place_and_cache_alone():
    row, q, pos, tab, slots, cache, weight = write_case(12, 6, 256, BF16, 4)
    lay = P.make_latent_layout(6, 256, cache.shape[0])
    g, gq, args = row.cuda(), q.cuda(), (pos.cuda(), tab.cuda(), slots.cuda())
    a, b = cache.cuda(), cache.cuda()
    out = torch.empty(12, 6, 64, dtype=BF16, device="cuda")
    P.pa_latent_write(g[:, :256], g[:, 256:320], gq[..., 128:], *args, out, a, lay)
    P.pa_latent_write(g[:, :256], g[:, 256:320], None, *args, None, b, lay)
    P.pa_latent_write(g[:, :256], g[:, 256:320], gq[..., 128:], *args, gq[..., 128:], b, lay)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(gq[..., 128:], out) and torch.equal(gq[..., :128].cpu(), q[..., :128])


# ---------------------------------------------------------------- absorbed attention

def absorbed(step, **kw):
    d = step.run(**kw)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == 0
    want, mag = step.want()
    check(d["out"], want, mag, step.dtype, step.logit_size(), step.latent + 64)
    return d


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("heads", [1, 5, 16, 17, 32, 40, 64, 128, 200])
def test_decode(heads, latent, dtype):
    """One token a request; lengths around pages, tiles and several of them."""
    absorbed(Step(heads, latent, [1] * 12, [1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 300, 777], dtype, seed=heads))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("heads,q_lens,seq_lens", [
    (16, [2, 1, 8, 3], [2, 70, 200, 64]), (3, [16, 5, 1], [16, 69, 130]), (32, [7], [400]), (64, [3, 2], [66, 2]),
    (128, [2, 5], [65, 100]), (1, [64, 1, 33], [64, 1, 97]), (20, [13, 16], [13, 1000])])
def test_few_tokens(heads, q_lens, seq_lens, latent, dtype):
    absorbed(Step(heads, latent, q_lens, seq_lens, dtype, seed=len(q_lens) + heads))


@pytest.mark.parametrize("heads,latent,n", [(16, 512, 1), (4, 256, 1), (32, 512, 3), (128, 512, 2), (64, 256, 5)])
def test_long(heads, latent, n):
    """Keys over many CTAs, joined."""
    absorbed(Step(heads, latent, [1] * n, [9000 - 1111 * i for i in range(n)], seed=n))


def test_many_requests():
    """More requests than a CTA has threads, of every length up to 90."""
    lens = [1 + i % 90 for i in range(500)]
    absorbed(Step(4, 256, [1] * 500, lens, seed=8))


def test_long_chunk():
    absorbed(Step(8, 512, [300, 40], [300, 640], seed=6))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_logits(dtype):
    """Logits of thousands, maxima that move from tile to tile."""
    step = Step(16, 256, [1, 1, 4], [500, 64, 300], dtype, seed=11, scale=1.0)
    step.q *= 8
    for r in range(3):  # keys that grow along the request
        n = int(step.seq_lens[r])
        pos = np.arange(n)
        at = (step.tables[r, pos // 16], pos % 16)
        step.cache[at] = (step.cache[at].float() * torch.linspace(0.1, 3, n)[:, None]).to(dtype)
    d = step.run()
    torch.cuda.synchronize()
    want, mag = step.want()
    if dtype == F32:
        check(d["out"], want, mag, dtype, step.logit_size(), 320)
    else:  # logits of thousands: the bound on a weight is above one; what is left is that a row is a mean of keys
        g = d["out"].double().cpu().numpy()
        assert np.isfinite(g).all()
        size = 2 * step.logit_size() * 1.4427 * 320 * 2.0 ** -24
        near = np.abs(g - want) <= mag * (2.0 ** -8 + 2 * np.expm1(size)) + np.abs(want) * 2.0 ** -8 * (1 + 2.0 ** -7)
        assert near.all()


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_scales(scale):
    absorbed(Step(8, 256, [1, 3], [200, 90], seed=12, scale=scale))


def test_results_repeat():
    step = Step(32, 512, [1] * 40 + [3] * 4, list(range(200, 2200, 50)) + [500] * 4, seed=13)
    d = step.run()
    first = d["out"].clone()
    for _ in range(3):
        d["out"].zero_()
        d["ws"].random_(0, 256)
        step.run(d)
        torch.cuda.synchronize()
        assert torch.equal(d["out"], first)


def test_rows_behind_the_step_stay():
    """out has rows behind the last request's in a padded batch: a second call's rows."""
    step = Step(16, 512, [1, 2], [50, 70], seed=14)
    d = step.gpu()
    whole = torch.full((10, 16, 512), 7.0, dtype=BF16, device="cuda")
    d["out"] = whole[:3]
    step.run(d)
    torch.cuda.synchronize()
    assert (whole[3:] == 7).all()
    want, mag = step.want()
    check(whole[:3], want, mag, BF16, step.logit_size(), 576)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bad_requests_are_skipped(dtype):
    """A length out of range leaves that request's rows, flags it and computes the others."""
    step = Step(16, 256, [1, 2, 1, 1], [40, 70, 30, 500], dtype, seed=15)
    want, mag = step.want()
    for r, bad in ((1, 1), (2, 0), (3, 501), (0, -5)):
        d = step.gpu()
        d["seq"][r] = bad
        step.run(d)
        torch.cuda.synchronize()
        assert int(d["status"].item()) == P.PA_DEV_LENGTHS
        rows = np.ones(5, bool)
        rows[step.starts[r]:step.starts[r + 1]] = False
        check(d["out"][torch.from_numpy(rows)], want[rows], mag[rows], dtype, step.logit_size(), 320)
        assert (d["out"][torch.from_numpy(~rows)] == 7).all()
    # a longer query than the bound
    d = step.run(max_q=1)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == P.PA_DEV_LENGTHS and (d["out"][1:3] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bad_starts_write_nothing(dtype):
    step = Step(16, 256, [1, 2, 1], [40, 70, 30], dtype, seed=16)
    for qsl in ([1, 1, 3, 4], [0, 1, 3, 5], [0, 3, 1, 4], [0, 1, 3, 3]):
        d = step.gpu()
        d["qsl"].copy_(torch.tensor(qsl, dtype=torch.int32))
        step.run(d)
        torch.cuda.synchronize()
        assert int(d["status"].item()) & P.PA_DEV_QSL
        assert (d["out"] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bad_blocks_read_as_zeros(dtype):
    step = Step(16, 256, [1, 1], [100, 40], dtype, seed=17)
    d = step.gpu()
    d["tables"][0, 2] = step.blocks + 3
    d["tables"][0, 4] = -7
    step.run(d)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == P.PA_DEV_BLOCK_RANGE
    for b in (2, 4):
        step.cache[step.tables[0, b]] = 0
    want, mag = step.want()
    check(d["out"], want, mag, dtype, step.logit_size(), 320)


def test_nan_stays_in_its_request():
    step = Step(16, 512, [1, 1, 1], [100, 130, 64], seed=18)
    step.cache[step.tables[1, 3], 5] = float("nan")
    d = step.run()
    torch.cuda.synchronize()
    assert d["out"][1].isnan().all()
    assert d["out"][[0, 2]].isfinite().all()


def test_infinite_logits():
    """A key whose logits are -inf has weight 0; one with +inf makes the row NaN."""
    step = Step(4, 256, [1, 1], [100, 100], F32, seed=19)
    for dtype in (F32, BF16):
        s = Step(4, 256, [1, 1], [100, 100], dtype, seed=19)
        s.q[:, :, 300] = 1.0
        s.cache[s.tables[0, 2], 3, 300] = float("-inf")  # in the key part: no value is infinite
        s.cache[s.tables[1, 2], 3, 300] = float("inf")
        d = s.run()
        torch.cuda.synchronize()
        with np.errstate(invalid="ignore"):
            want, mag = s.want()
        assert d["out"][1].isnan().all()
        s.cache[~s.cache.isfinite() & ~s.cache.isnan()] = 0
        check(d["out"][:1], want[:1], mag[:1], dtype, s.logit_size(), 320)


def test_streams_and_graph():
    """Two streams with workspaces of their own, a captured step replayed on new data."""
    steps = [Step(32, 512, [1] * 30, list(range(100, 3100, 100)), seed=s) for s in (20, 21)]
    ds = [s.gpu() for s in steps]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, d, st in zip(steps, ds, streams):
            s.run(d, stream=st)
    torch.cuda.synchronize()
    for s, d in zip(steps, ds):
        want, mag = s.want()
        check(d["out"], want, mag, BF16, s.logit_size(), 576)
    d = ds[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps[0].run(d)
    d["q"].copy_(steps[1].q)
    d["seq"].copy_(torch.from_numpy(np.maximum(1, steps[0].seq_lens - 37)))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    steps[0].q, steps[0].seq_lens = steps[1].q, np.maximum(1, steps[0].seq_lens - 37)
    want, mag = steps[0].want()
    check(d["out"], want, mag, BF16, steps[0].logit_size(), 576)


@pytest.mark.parametrize("seq_lens", [[40, 7, 130], [900, 130, 2000]])
def test_lengths_of_the_kernel_before(seq_lens):
    """A captured loop of steps whose lengths the kernel right before each call moves on."""
    step = Step(16, 256, [1] * 3, seq_lens, seed=40)
    d = step.gpu()
    outs = [torch.empty_like(d["out"]) for _ in range(6)]
    step.run(d)  # (takes the workspace)
    d["seq"] -= len(outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for out in outs:
            d["seq"].add_(1)
            step.run({**d, "out": out}, max_q=1, max_s=max(seq_lens))
    graph.replay()
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        step.seq_lens = np.asarray(seq_lens) - len(outs) + 1 + i
        want, mag = step.want()
        check(out, want, mag, BF16, step.logit_size(), 320)


def test_cache_past_4_gib():
    """Slots whose bytes lie past 32 bits: written, read back and attended over."""
    heads, r, n = 4, 512, 300
    blocks = (5 << 30) // (16 * 576 * 2)
    cache = torch.empty(blocks, 16, r + 64, dtype=BF16, device="cuda")
    small = Step(heads, r, [1, 2], [n, 40], seed=30)
    lay = P.latent_layout_of(cache, heads)
    # the small cache's blocks, written far up by their rows
    high = blocks - 1 - torch.arange(small.blocks)
    rows = small.cache.flatten(0, 1).nan_to_num()
    slots = (high[:, None] * 16 + torch.arange(16)).flatten().cuda()
    tab = torch.from_numpy(O.table(1, 64)).float().cuda()  # position 0 turns nothing
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = rows.cuda()
    P.pa_latent_write(g[:, :r], g[:, r:], None, torch.zeros(len(rows), dtype=torch.int64, device="cuda"), tab, slots, None, cache,
                      lay, status=status)
    c, k = torch.empty(len(rows), r, dtype=BF16, device="cuda"), torch.empty(len(rows), 64, dtype=BF16, device="cuda")
    P.pa_latent_read(cache, slots, c, k, lay, status)
    d = small.gpu()
    d["cache"] = cache
    d["tables"] = torch.where(d["tables"] >= 0, blocks - 1 - d["tables"], d["tables"])
    d["status"] = status
    small.run(d, layout=lay)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(torch.cat([c, k], -1).cpu(), rows)
    want, mag = small.want()
    check(d["out"], want, mag, BF16, small.logit_size(), 576)


def test_same_cache_two_steps_at_once():
    """Two steps on two streams read one cache, each with its workspace and its head count."""
    a = Step(16, 512, [1] * 20, list(range(50, 1050, 50)), seed=31)
    b = Step(64, 512, [1] * 20, list(range(50, 1050, 50)), seed=31)
    b.cache, b.tables = a.cache, a.tables
    da, db = a.gpu(), b.gpu()
    db["cache"] = da["cache"]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(da, stream=s1)
        b.run(db, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    for st, d in ((a, da), (b, db)):
        want, mag = st.want()
        check(d["out"], want, mag, BF16, st.logit_size(), 576)
