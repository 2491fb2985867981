"""Expanded latent attention, and the two forms together."""
import numpy as np
import pytest
import torch

import paged_kv_attention_04_gb300 as P
from latent_cases import check
from oracle import latent as O

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_attention_04_gb300 import build
    build.build()
    P.lib()


class Prompts:
    """Ragged requests of q_lens rows over seq_lens keys; keys and values are slices of one projection."""

    def __init__(self, heads, size, q_lens, seq_lens, dtype=BF16, seed=0, scale=None, spare=0):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.size, self.dtype = heads, size, dtype
        self.q_lens, self.seq_lens = np.asarray(q_lens), np.asarray(seq_lens)
        self.starts, self.kv_starts = (np.concatenate([[0], np.cumsum(x)]) for x in (q_lens, seq_lens))
        t, tk = int(self.starts[-1]), int(self.kv_starts[-1])
        self.q = torch.randn(t + spare, heads, size + 64, generator=g).to(dtype)
        self.kv = torch.randn(tk + spare, heads, 2 * size, generator=g).to(dtype)
        self.rope = torch.randn(tk + spare, 128, generator=g).to(dtype)
        self.tokens, self.keys = t, tk
        self.scale = scale if scale is not None else (size + 64) ** -0.5

    def gpu(self):
        i32 = lambda x: torch.from_numpy(x.astype(np.int32)).cuda()  # noqa: E731
        kv = self.kv.cuda()
        d = self.size
        return dict(q=self.q.cuda()[:self.tokens], k=kv[:self.keys, :, :d], v=kv[:self.keys, :, d:],
                    kr=self.rope.cuda()[:self.keys, 64:], qsl=i32(self.starts), kvsl=i32(self.kv_starts),
                    out=torch.full((self.tokens, self.heads, d), 7.0, dtype=self.dtype, device="cuda"),
                    status=torch.zeros(1, dtype=torch.int32, device="cuda"))

    def run(self, d=None, max_q=None, max_kv=None, stream=None):
        d = d or self.gpu()
        P.pa_expanded_forward(d["q"], d["k"], d["kr"], d["v"], d["qsl"], d["kvsl"], max_q or int(self.q_lens.max()),
                              max_kv or int(self.seq_lens.max()), self.scale, d["out"], status=d["status"], stream=stream)
        return d

    def want(self):
        f = lambda x: x.double().numpy()  # noqa: E731
        d = self.size
        return O.expanded(f(self.q[:self.tokens]), f(self.kv[:self.keys, :, :d]), f(self.rope[:self.keys, 64:]),
                          f(self.kv[:self.keys, :, d:]), self.starts, self.kv_starts, self.scale)

    def logit_size(self):
        q = self.q[:self.tokens].double().nan_to_num().abs()
        k = torch.cat([self.kv[:self.keys, :, :self.size].double().nan_to_num().abs(),
                       self.rope[:self.keys, None, 64:].double().nan_to_num().abs().expand(-1, self.heads, -1)], -1)
        return max(float((q[:, h] @ k[:, h].T).max()) for h in range(self.heads)) * abs(self.scale)

    def check(self, d, rows=None):
        want, mag = self.want()
        rows = slice(None) if rows is None else rows
        return check(d["out"][rows], want[rows], mag[rows], self.dtype, self.logit_size(), self.size + 64)


def attend(step, **kw):
    d = step.run(**kw)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == 0
    step.check(d)
    return d


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [64, 128])
@pytest.mark.parametrize("heads,q_lens,seq_lens", [
    (1, [1], [1]), (3, [1, 2, 17], [1, 2, 17]), (2, [127, 128, 129], [127, 128, 129]), (5, [255, 256, 257], [255, 256, 257]),
    (4, [1, 1, 1], [1, 128, 300]), (2, [64, 300], [640, 301]), (1, [200], [1111]), (16, [33, 1, 90], [33, 200, 128])])
def test_shapes(heads, q_lens, seq_lens, size, dtype):
    attend(Prompts(heads, size, q_lens, seq_lens, dtype, seed=heads))


def test_long_prompts():
    """Many tiles a unit, many units a CTA: every place of the ring, units of several requests in turn."""
    attend(Prompts(8, 128, [1500, 700, 1, 1024], [1500, 2300, 3000, 1024], seed=1))
    attend(Prompts(40, 128, [260, 300], [260, 1300], seed=2))
    attend(Prompts(40, 64, [900, 300], [900, 1300], seed=3))


@pytest.mark.parametrize("heads,size,q_lens,seq_lens", [
    (1, 128, [300], [5000]), (3, 64, [700, 1], [2100, 3000]), (2, 128, [130, 257, 40], [1500, 257, 4100]),
    (24, 128, [1000], [1000]), (16, 64, [900], [3700])])
def test_cut_units(heads, size, q_lens, seq_lens):
    """Few units of many tiles, in pieces over the SMs; with a caller's workspace, filled with anything, too."""
    step = Prompts(heads, size, q_lens, seq_lens, seed=20)
    need = P.pa_expanded_workspace_size(heads, size, step.tokens, max(seq_lens)) if max(seq_lens) >= 1024 else 0
    assert (need > 0) == (max(seq_lens) >= 1024)
    d = attend(step)
    first = d["out"].clone()
    ws = torch.randint(0, 256, (max(need, 256),), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        d["out"].zero_()
        P.pa_expanded_forward(d["q"], d["k"], d["kr"], d["v"], d["qsl"], d["kvsl"], max(q_lens), max(seq_lens), step.scale,
                              d["out"], workspace=ws, status=d["status"])
        torch.cuda.synchronize()
        assert torch.equal(d["out"], first) and int(d["status"].item()) == 0


def test_many_requests():
    n = [1 + i % 40 for i in range(500)]
    attend(Prompts(2, 64, n, [x + 3 * (i % 7) for i, x in enumerate(n)], seed=4))


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_scales(scale):
    step = Prompts(2, 128, [40, 150], [140, 150], seed=5, scale=scale)
    attend(step)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_neighbours_nan_stays_theirs(dtype):
    """Rows of other requests and rows behind the last key are NaN: no trace of them."""
    step = Prompts(3, 128, [20, 50, 30], [100, 50, 230], dtype, seed=6, spare=200)
    step.kv[100:150] = float("nan")
    step.rope[100:150] = float("nan")
    step.q[20:70] = float("nan")
    step.q[100:] = float("nan")
    step.kv[380:], step.rope[380:] = float("nan"), float("nan")
    d = step.run()
    torch.cuda.synchronize()
    rows = np.r_[0:20, 70:100]
    assert d["out"][20:70].isnan().all()
    step.q.nan_to_num_(0), step.kv.nan_to_num_(0), step.rope.nan_to_num_(0)
    step.check(d, rows)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bad_inputs(dtype):
    step = Prompts(2, 64, [20, 50, 30], [100, 50, 230], dtype, seed=7)
    for over, bad, flag in ((dict(max_q=40), [1], P.PA_DEV_LENGTHS), (dict(max_kv=200), [2], P.PA_DEV_LENGTHS)):
        d = step.run(**over)
        torch.cuda.synchronize()
        assert int(d["status"].item()) == flag
        rows = np.concatenate([np.arange(step.starts[r], step.starts[r + 1]) for r in range(3) if r not in bad])
        step.check(d, rows)
        assert (d["out"][step.starts[bad[0]]:step.starts[bad[0] + 1]] == 7).all()
    # more rows than keys
    d = step.gpu()
    d["kvsl"].copy_(torch.tensor([0, 120, 140, 380]))
    step.run(d)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == P.PA_DEV_LENGTHS and (d["out"][20:70] == 7).all()
    for qsl, kvsl in (([0, 20, 70, 99], None), ([1, 20, 70, 100], None), ([0, 70, 20, 100], None),
                      (None, [0, 100, 150, 379]), (None, [0, 150, 100, 380])):
        d = step.gpu()
        if qsl:
            d["qsl"].copy_(torch.tensor(qsl))
        if kvsl:
            d["kvsl"].copy_(torch.tensor(kvsl))
        step.run(d)
        torch.cuda.synchronize()
        assert int(d["status"].item()) & P.PA_DEV_QSL and (d["out"] == 7).all()


def test_layouts():
    """Every operand contiguous, and heads before tokens."""
    step = Prompts(6, 128, [130, 40], [200, 40], seed=8)
    d = step.gpu()
    for k in "qkv":
        d[k] = d[k].contiguous()
    d["kr"] = d["kr"].contiguous()
    a = step.run(d)["out"].clone()
    for k in "qkv":
        d[k] = d[k].transpose(0, 1).contiguous().transpose(0, 1)
    b = step.run(d)["out"]
    torch.cuda.synchronize()
    step.check(d)
    assert torch.equal(a, b)


def test_repeats_streams_and_graph():
    steps = [Prompts(32, 128, [300, 700], [300, 1900], seed=s) for s in (9, 10)]
    ds = [s.gpu() for s in steps]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, d, st in zip(steps, ds, streams):
            s.run(d, stream=st)
    torch.cuda.synchronize()
    first = [d["out"].clone() for d in ds]
    for s, d in zip(steps, ds):
        s.check(d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps[0].run(ds[0])
    for k in ("q", "k", "v", "kr"):
        ds[0][k].copy_(ds[1][k])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ds[0]["out"], first[1])


@pytest.mark.parametrize("q_lens,seq_lens", [([3, 150], [40, 150]), ([200], [2500])])
def test_starts_of_the_kernel_before(q_lens, seq_lens):
    """Captured calls whose starts the kernel right before each writes."""
    step = Prompts(2, 64, q_lens, seq_lens, seed=13)
    d = step.gpu()
    want = step.run()["out"]
    zero, outs = torch.zeros_like(d["qsl"]), [torch.empty_like(d["out"]) for _ in range(4)]
    q0, k0 = d["qsl"].clone(), d["kvsl"].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for out in outs:
            torch.add(k0, zero, out=d["kvsl"])
            torch.add(q0, zero, out=d["qsl"])
            step.run({**d, "out": out})
            d["qsl"].zero_()
            d["kvsl"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    step.check({"out": want})
    assert int(d["status"].item()) == 0
    for out in outs:
        assert torch.equal(out, want)


def test_cut_units_on_another_stream():
    """The workspace that the call takes itself belongs to the stream it runs on: memory that work on the current
    stream still reads is not given to it."""
    step = Prompts(4, 128, [300], [3000], seed=12)
    want, mag = step.want()
    side = torch.cuda.Stream()
    d = step.gpu()
    torch.cuda.synchronize()
    need = P.pa_expanded_workspace_size(4, 128, 300, 3000)
    for handle in (side, side.cuda_stream):
        busy = torch.full((need // 4,), 3.0, device="cuda")
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            big = (big @ big).clamp(-1, 1)
        kept = busy + big[0, 0] * 0  # read late on the current stream
        del busy
        step.run(d, stream=handle)
        torch.cuda.synchronize()
        assert (kept == 3).all()
        check(d["out"], want, mag, BF16, step.logit_size(), 192)


def test_layer_step():
    """A layer as it runs: prompts' latents appended (norm, rotation), read back and expanded for the prompts'
    attention, then two decode steps over the cache in the absorbed form; each against the 64-bit layer."""
    heads, r, d, lens, steps = 4, 256, 64, [37, 100, 5], 2
    g = torch.Generator(device="cuda").manual_seed(11)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    wk, wv = rand(heads, r, d) * r ** -0.5, rand(heads, r, d) * r ** -0.5
    weight = 1 + 0.1 * rand(r)
    tab = torch.from_numpy(O.table(200, 64)).float().cuda()
    nb = 8
    tables = torch.randperm(3 * nb + 4, generator=torch.Generator().manual_seed(1))[:3 * nb].view(3, nb).cuda()
    cache = torch.full((3 * nb + 4, 16, r + 64), float("nan"), dtype=BF16, device="cuda")
    lay, scale = P.latent_layout_of(cache, heads), (d + 64) ** -0.5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rows64 = [torch.zeros(0, r + 64, dtype=torch.float64, device="cuda") for _ in lens]  # what each request's slots hold

    def new_tokens(counts, done):
        pos = torch.cat([torch.arange(b, b + n) for n, b in zip(counts, done)]).cuda()
        req = torch.repeat_interleave(torch.arange(3), torch.tensor(counts)).cuda()
        slots = tables[req, pos // 16] * 16 + pos % 16
        n = sum(counts)
        return pos, slots, rand(n, r + 64), rand(n, heads, d + 64)

    def turn(x, pos):
        return torch.from_numpy(O.rotate(x.double().cpu().numpy(), tab.double().cpu().numpy(), pos.cpu().numpy(), True)).cuda()

    def append(counts, pos, slots, row, q, q_out):
        P.pa_latent_write(row[:, :r], row[:, r:], q[..., d:], pos, tab, slots, q_out, cache, lay, norm_weight=weight, pairs=True,
                          status=status)
        a = 0
        for i, n in enumerate(counts):  # the rows as held: rounded to bf16
            rows64[i] = torch.cat([rows64[i], cache.flatten(0, 1)[slots[a:a + n]].double()])
            a += n
        # ... which are what the definition gives, to a rounding
        c = torch.from_numpy(O.rms_norm(row[:, :r].double().cpu().numpy(), weight.double().cpu().numpy(), 1e-6)).cuda()
        held = cache.flatten(0, 1)[slots].double()
        exact = torch.cat([c, turn(row[:, r:], pos)], -1)
        assert bool(((held - exact).abs() <= exact.abs() * 2.0 ** -8 * (1 + 2.0 ** -6) + 2.0 ** -20).all())

    # the prompts
    pos, slots, row, q = new_tokens(lens, [0, 0, 0])
    append(lens, pos, slots, row, q, q[..., d:])  # (q's parts rotated in place)
    q_plain = q.clone()
    c, kr = torch.empty(len(slots), r, dtype=BF16, device="cuda"), torch.empty(len(slots), 64, dtype=BF16, device="cuda")
    P.pa_latent_read(cache, slots, c, kr, lay, status)
    kv = torch.einsum("tr,hrd->thd", c.float(), torch.cat([wk, wv], -1).float()).to(BF16)
    starts = i32(np.concatenate([[0], np.cumsum(lens)]))
    out = torch.empty(sum(lens), heads, d, dtype=BF16, device="cuda")
    P.pa_expanded_forward(q_plain, kv[..., :d], kr, kv[..., d:], starts, starts, max(lens), max(lens), scale, out, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0

    def near(got, q_turned, counts):
        """Keys and values (or queries and outputs) are rounded to bf16 on the way, and so are the rotated
        queries: relative errors of 2^-8 in factors of a logit move a weight by up to the sum of
        |q k| scale 2^-8 each; here that sum is below 12, three such factors meet in a logit."""
        a, outs, mags = 0, [], []
        for i, n in enumerate(counts):
            cc, kk = rows64[i][:, :r], rows64[i][:, r:]
            kn, v = (torch.einsum("tr,hrd->thd", cc, w.double()) for w in (wk, wv))
            o = O.expanded(*(x.cpu().numpy() for x in (q_turned[a:a + n].double(), kn, kk, v)), [0, n], [0, len(cc)], scale)
            outs.append(o[0])
            mags.append(o[1])
            a += n
        want, mag = np.concatenate(outs), np.concatenate(mags)
        assert (np.abs(got.double().cpu().numpy() - want) <= mag * (2 * 12 * 3 + 4) * 2.0 ** -8).all()
        rel = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
        # roundings of 2^-9 rms each, a handful of them
        assert rel < 8 * 2.0 ** -9, rel

    near(out, q_plain, lens)
    # decodes
    done = list(lens)
    for _ in range(steps):
        pos, slots, row, q = new_tokens([1, 1, 1], done)
        q_abs = torch.empty(3, heads, r + 64, dtype=BF16, device="cuda")
        append([1, 1, 1], pos, slots, row, q, q_abs[..., r:])
        q_abs[..., :r] = torch.einsum("thd,hrd->thr", q[..., :d].float(), wk.float())
        done = [x + 1 for x in done]
        o = torch.empty(3, heads, r, dtype=BF16, device="cuda")
        ws = P.alloc_latent_workspace(lay, 3, 3, 1, max(done))
        P.pa_latent_forward(q_abs, cache, tables.to(torch.int32), i32(done), i32([0, 1, 2, 3]), 1, max(done), scale, o, ws, lay,
                            status)
        got = torch.einsum("thr,hrd->thd", o.float(), wv.float())
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        near(got, torch.cat([q[..., :d], q_abs[..., r:]], -1), [1, 1, 1])
