"""What the rotating write and the latent-attention calls refuse, at the C boundary and in the binding.
Nothing runs on a GPU: the C calls return before a launch, the binding's launch is replaced."""
import ctypes

import pytest
import torch

import paged_kv_attention_04_gb300 as P
from paged_kv_attention_04_gb300 import binding

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_04_gb300 import build
    build.build()
    return P.lib()


# ---------------------------------------------------------------- the C boundary

def rope(**over):
    a = dict(positions=256, cos_sin=256, max_position=100, rope_size=64, style=0)
    a.update(over)
    return P.pa_rope(a["positions"], a["cos_sin"], a["max_position"], a["rope_size"], a["style"])


BAD_ROPES = [dict(positions=None), dict(cos_sin=None), dict(positions=260), dict(cos_sin=264), dict(max_position=0),
             dict(rope_size=0), dict(rope_size=24), dict(style=2)]


def rope_write(lib, lay=None, r=None, **over):
    lay = lay or P.make_layout(8, 2, 64, 4, BF16)
    a = dict(q=256, qs=512, k=256, ks=128, v=256, vs=128, slots=256, n=3, qo=512, kc=256, vc=256, status=None)
    a.update(over)
    return lib.pa_rope_cache_write(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], r or rope(), a["slots"], a["n"],
                                   a["qo"], a["kc"], a["vc"], lay, a["status"], None)


def test_rope_write_refusals(lib):
    assert rope_write(lib, n=0) == P.PA_OK
    for r in BAD_ROPES + [dict(rope_size=80)]:
        assert rope_write(lib, r=rope(**r)) == P.PA_ERR_INVALID, r
        assert P.last_error()
    for over in (dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(k=264), dict(q=264), dict(qo=520),
                 dict(slots=260), dict(q=None), dict(qo=None), dict(ks=120), dict(vs=132), dict(qs=510), dict(n=-1),
                 dict(status=258), dict(qo=256, qs=520), dict(n=1 << 28)):
        assert rope_write(lib, **over) == P.PA_ERR_INVALID, over
    assert rope_write(lib, lay=P.make_layout(8, 2, 96, 4, BF16)) == P.PA_ERR_UNSUPPORTED
    assert lib.pa_rope_cache_write(256, 512, 256, 128, 256, 128, None, 256, 1, 512, 256, 256,
                                   P.make_layout(8, 2, 64, 4, BF16), None, None) == P.PA_ERR_INVALID


def latent(**over):
    a = dict(num_heads=16, latent_size=512, num_blocks=10, dtype=BF16, rope_size=64, block_size=16)
    a.update(over)
    return P.make_latent_layout(**a)


BAD_LATENTS = [(dict(num_heads=0), P.PA_ERR_INVALID), (dict(num_heads=257), P.PA_ERR_UNSUPPORTED),
               (dict(latent_size=384), P.PA_ERR_UNSUPPORTED), (dict(rope_size=32), P.PA_ERR_UNSUPPORTED),
               (dict(block_size=32), P.PA_ERR_UNSUPPORTED), (dict(num_blocks=0), P.PA_ERR_INVALID),
               (dict(dtype=P.PA_FP8_E4M3), P.PA_ERR_INVALID), (dict(dtype=7), P.PA_ERR_INVALID)]


def latent_write(lib, lay=None, r=None, **over):
    a = dict(c=256, cs=576, k=256, ks=576, w=256, eps=1e-6, q=256, qs=16 * 192, qh=192, slots=256, n=3, qo=512,
             os=16 * 576, oh=576, cache=256, status=None)
    a.update(over)
    return lib.pa_latent_write(a["c"], a["cs"], a["k"], a["ks"], a["w"], a["eps"], a["q"], a["qs"], a["qh"], r or rope(),
                               a["slots"], a["n"], a["qo"], a["os"], a["oh"], a["cache"], lay or latent(), a["status"], None)


def test_latent_write_refusals(lib):
    assert latent_write(lib, n=0) == P.PA_OK
    for over, code in BAD_LATENTS:
        assert latent_write(lib, lay=latent(**over)) == code, over
        assert P.last_error()
    for r in BAD_ROPES + [dict(rope_size=48)]:
        assert latent_write(lib, r=rope(**r)) == P.PA_ERR_INVALID, r
    for over in (dict(c=None), dict(k=None), dict(slots=None), dict(cache=None), dict(c=264), dict(k=258), dict(w=264),
                 dict(cache=264), dict(q=264), dict(qo=520), dict(slots=260), dict(status=2), dict(cs=504), dict(ks=60),
                 dict(cs=577), dict(qs=16 * 192 + 4), dict(qh=60), dict(qs=15 * 192), dict(oh=570), dict(os=100),
                 dict(q=None), dict(qo=None), dict(qo=256), dict(n=-1), dict(eps=float("nan")), dict(eps=-1.0)):
        assert latent_write(lib, **over) == P.PA_ERR_INVALID, over


def test_latent_read_refusals(lib):
    call = lambda cache=256, slots=256, n=3, c=256, k=256, lay=None, status=None: lib.pa_latent_read(  # noqa: E731
        cache, slots, n, c, k, lay or latent(), status, None)
    assert call(n=0) == P.PA_OK
    for over, code in BAD_LATENTS:
        assert call(lay=latent(**over)) == code, over
    for over in (dict(cache=None), dict(slots=None), dict(c=None), dict(k=None), dict(cache=264), dict(c=264), dict(k=264),
                 dict(slots=4), dict(status=2), dict(n=-1)):
        assert call(**over) == P.PA_ERR_INVALID, over


def latent_forward(lib, lay=None, **over):
    a = dict(q=256, cache=256, bt=256, maxb=4, sl=256, qsl=256, B=2, T=2, maxq=1, maxs=64, scale=0.1, out=256, ws=256,
             wsb=1 << 30, status=None)
    a.update(over)
    return lib.pa_latent_forward(a["q"], a["cache"], a["bt"], a["maxb"], a["sl"], a["qsl"], a["B"], a["T"], a["maxq"],
                                 a["maxs"], a["scale"], a["out"], a["ws"], a["wsb"], lay or latent(), a["status"], None)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_latent_forward_refusals(lib, dtype):
    assert latent_forward(lib, latent(dtype=dtype), B=0, T=0) == P.PA_OK
    for over, code in BAD_LATENTS:
        assert latent_forward(lib, lay=latent(**over)) == code, over
        assert lib.pa_latent_workspace_size(latent(**over), 2, 2, 1, 64) == 0 and P.last_error()
    for over in (dict(q=None), dict(cache=None), dict(bt=None), dict(sl=None), dict(qsl=None), dict(out=None), dict(ws=None),
                 dict(q=264), dict(cache=264), dict(out=264), dict(bt=258), dict(sl=257), dict(qsl=258), dict(ws=272),
                 dict(wsb=1024), dict(maxb=3), dict(T=1), dict(maxq=0), dict(maxs=0), dict(B=-1), dict(scale=float("inf")),
                 dict(status=3), dict(T=1 << 30)):
        assert latent_forward(lib, latent(dtype=dtype), **over) == P.PA_ERR_INVALID, over
        assert P.last_error()


def test_latent_workspace(lib):
    size = lambda lay, *a: P.pa_latent_workspace_size(lay, *a)  # noqa: E731
    a, b, c = (size(latent(num_heads=h), 4, 4, 1, 4096) for h in (16, 32, 64))
    assert 0 < a < b < c and c % 256 == 0
    assert size(latent(num_heads=16), 4, 16, 4, 4096) == c       # rows of a request: heads x tokens
    assert size(latent(num_heads=16), 4, 4, 1, 1 << 20) == a     # not the length
    with pytest.raises(P.PaError, match="latent_size"):
        size(latent(latent_size=100), 1, 1, 1, 16)
    with pytest.raises(P.PaError, match="negative"):
        size(latent(), 1, -1, 1, 16)


def expanded(lib, over_lay=(), **over):
    lay = dict(num_heads=4, head_size=128, rope_size=64, dtype=P.PA_BF16, q_stride=768, q_head_stride=192, k_stride=1024,
               k_head_stride=256, kr_stride=64, v_stride=1024, v_head_stride=256)
    lay.update(over_lay)
    a = dict(q=256, k=256, kr=256, v=256, qsl=256, kvsl=256, B=2, T=4, Tk=10, maxq=3, maxkv=8, scale=0.1, out=256, ws=None,
             wsb=0, status=None)
    a.update(over)
    return lib.pa_expanded_forward(a["q"], a["k"], a["kr"], a["v"], a["qsl"], a["kvsl"], a["B"], a["T"], a["Tk"], a["maxq"],
                                   a["maxkv"], a["scale"], a["out"], a["ws"], a["wsb"], P.pa_expanded_layout(**lay),
                                   a["status"], None)


@pytest.mark.parametrize("dtype", [P.PA_BF16, P.PA_F32])
def test_expanded_refusals(lib, dtype):
    assert expanded(lib, dict(dtype=dtype), B=0, T=0) == P.PA_OK
    for lay, code in ((dict(head_size=96), P.PA_ERR_UNSUPPORTED), (dict(rope_size=32), P.PA_ERR_UNSUPPORTED),
                      (dict(num_heads=300), P.PA_ERR_UNSUPPORTED), (dict(num_heads=0), P.PA_ERR_INVALID),
                      (dict(dtype=P.PA_INT4), P.PA_ERR_INVALID), (dict(q_stride=766, dtype=dtype), P.PA_ERR_INVALID),
                      (dict(k_head_stride=0, dtype=dtype), P.PA_ERR_INVALID), (dict(kr_stride=-64, dtype=dtype), P.PA_ERR_INVALID),
                      (dict(v_stride=1 << 41, dtype=dtype), P.PA_ERR_INVALID)):
        assert expanded(lib, lay) == code, lay
        assert P.last_error()
    for over in (dict(q=None), dict(k=None), dict(kr=None), dict(v=None), dict(qsl=None), dict(kvsl=None), dict(out=None),
                 dict(q=264), dict(k=264), dict(kr=264), dict(v=264), dict(out=264), dict(qsl=2), dict(kvsl=2), dict(T=1),
                 dict(Tk=3), dict(maxq=0), dict(maxkv=0), dict(scale=float("nan")), dict(status=2), dict(B=-1), dict(ws=272)):
        assert expanded(lib, dict(dtype=dtype), **over) == P.PA_ERR_INVALID, over
    assert lib.pa_expanded_forward(256, 256, 256, 256, 256, 256, 1, 1, 1, 1, 1, 0.1, 256, None, 0, None, None,
                                   None) == P.PA_ERR_INVALID


def test_expanded_workspace(lib):
    size = P.pa_expanded_workspace_size
    assert size(32, 128, 2048, 8192) > size(32, 64, 2048, 8192) > 0
    assert size(32, 128, 2048, 100) == 0            # short
    assert size(32, 128, 1 << 17, 8192) == 0        # many units
    assert size(32, 128, 2048, 8192, dtype=F32) == 0
    with pytest.raises(P.PaError, match="head_size"):
        size(32, 100, 2048, 8192)
    need = size(4, 128, 100, 4096)
    assert expanded(lib, T=100, Tk=4096, maxq=100, maxkv=4096, ws=256, wsb=need - 1) == P.PA_ERR_INVALID
    assert "workspace" in P.last_error()


# ---------------------------------------------------------------- the binding

def test_host_tensors_are_refused():
    z = lambda *s, t=BF16: torch.zeros(*s, dtype=t)  # noqa: E731
    i64, i32 = torch.zeros(1, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    lay, kc = P.make_layout(2, 1, 64, 2, BF16), z(2, 16, 1, 64)
    lat, cache = P.make_latent_layout(2, 256, 2), z(2, 16, 320)
    for call in (lambda: P.pa_rope_cache_write(z(1, 2, 64), z(1, 1, 64), z(1, 1, 64), i64, z(4, 64, t=F32), i64, z(1, 2, 64), kc,
                                               kc, lay),
                 lambda: P.pa_latent_write(z(1, 256), z(1, 64), None, i64, z(4, 64, t=F32), i64, None, cache, lat),
                 lambda: P.pa_latent_read(cache, i64, z(1, 256), z(1, 64), lat),
                 lambda: P.pa_latent_forward(z(1, 2, 320), cache, i32[None], i32[:1], i32, 1, 32, 1.0, z(1, 2, 256), z(64), lat),
                 lambda: P.pa_expanded_forward(z(1, 2, 192), z(1, 2, 128), z(1, 64), z(1, 2, 128), i32, i32, 1, 1, 1.0,
                                               z(1, 2, 128))):
        with pytest.raises(P.PaError, match="not a CUDA tensor"):
            call()


@pytest.fixture
def launched(monkeypatch, lib):
    calls = []
    monkeypatch.setattr(binding, "_device", lambda name, t: -1)  # (a host tensor's)
    monkeypatch.setattr(binding, "_launch", lambda fn, dev, stream, *args: calls.append(args))
    return calls


T, HQ, HKV, D, NB = 3, 4, 2, 64, 4


def rope_args(dtype=BF16, cache=None, **over):
    lay = P.make_layout(HQ, HKV, D, NB, dtype, cache_dtype=cache)
    held = dtype if cache is None else torch.uint8
    z = lambda *s, t=dtype: torch.zeros(*s, dtype=t)  # noqa: E731
    a = dict(q=z(T, HQ, D), k=z(T, HKV, D), v=z(T, HKV, D), positions=torch.zeros(T, dtype=torch.int64),
             cos_sin=z(9, 64, t=F32), slot_mapping=torch.zeros(T, dtype=torch.int64), q_out=z(T, HQ, D),
             k_cache=z(*P.cache_shape(lay), t=held), v_cache=z(*P.cache_shape(lay), t=held), layout=lay)
    a.update(over)
    return a


@pytest.mark.parametrize("dtype,cache", [(BF16, None), (F32, None), (BF16, P.PA_FP8_E4M3), (BF16, P.PA_INT4)])
def test_binding_rope_write(launched, dtype, cache):
    other = F32 if dtype == BF16 else BF16
    z = lambda *s, t=dtype: torch.zeros(*s, dtype=t)  # noqa: E731
    i64 = lambda n: torch.zeros(n, dtype=torch.int64)  # noqa: E731
    for over, match in ((dict(k=z(T, HKV, D, t=other)), "k is"), (dict(v=z(T - 1, HKV, D)), "v is"),
                        (dict(q=z(T, HQ + 1, D)), "q is"), (dict(q_out=z(T, HQ * D)), "q_out is"),
                        (dict(q_out=z(T, HQ, 2 * D)[..., :D]), "q_out is not contiguous"),
                        (dict(k=z(T, D, HKV).transpose(1, 2)), "must be contiguous"),
                        (dict(v=z(T, HKV, 2 * D)[..., :D]), "must be contiguous"),
                        (dict(positions=i64(T).int()), "positions is"), (dict(positions=i64(T - 1)), "positions for"),
                        (dict(slot_mapping=i64(T).int()), "slot_mapping is"), (dict(slot_mapping=i64(T - 1)), "slots for"),
                        (dict(cos_sin=z(9, 64, t=torch.float64)), "cos_sin is"), (dict(cos_sin=z(9, 128, t=F32)[:, :64]), "cos_sin"),
                        (dict(cos_sin=z(64, t=F32)), "cos_sin is"), (dict(q=None), "both be given"), (dict(q_out=None), "both be given"),
                        (dict(k_cache=z(NB, 16, HKV, D, t=torch.float64)), "k_cache is"), (dict(v_cache=z(NB - 1, 16, HKV, D)), "v_cache is"),
                        (dict(status=i64(1)), "status is")):
        with pytest.raises(P.PaError, match=match):
            P.pa_rope_cache_write(**rope_args(dtype, cache, **over))
    assert not launched
    P.pa_rope_cache_write(**rope_args(dtype, cache))
    P.pa_rope_cache_write(**rope_args(dtype, cache, q=None, q_out=None))
    # slices of one projection, and arrays with numbers to spare
    qkv = z(T, (HQ + 2 * HKV) * D)
    q, k, v = (x.unflatten(-1, (-1, D)) for x in qkv.split([HQ * D, HKV * D, HKV * D], -1))
    P.pa_rope_cache_write(**rope_args(dtype, cache, q=q, k=k, v=v, positions=i64(T + 2), slot_mapping=i64(T + 2)))
    row = (HQ + 2 * HKV) * D
    assert [(a[1], a[3], a[5], a[8]) for a in launched] == [(HQ * D, HKV * D, HKV * D, T), (0, HKV * D, HKV * D, T), (row, row, row, T)]


def test_binding_latent(launched):
    h, r, nb, b = 4, 256, 3, 2
    z = lambda *s, t=BF16: torch.zeros(*s, dtype=t)  # noqa: E731
    i64, i32 = (lambda n: torch.zeros(n, dtype=torch.int64)), (lambda *s: torch.zeros(*s, dtype=torch.int32))
    lay, cache = P.make_latent_layout(h, r, nb), z(nb, 16, r + 64)
    write = lambda **o: P.pa_latent_write(**{**dict(c=z(T, r), k_rope=z(T, 64), q=z(T, h, 64), positions=i64(T),  # noqa: E731
                                                    cos_sin=z(9, 64, t=F32), slot_mapping=i64(T), q_out=z(T, h, 64),
                                                    cache=cache, layout=lay), **o})
    for o, match in ((dict(c=z(T, r + 8)), "c is"), (dict(k_rope=z(T, 32)), "k_rope is"), (dict(q=z(T, h + 1, 64)), "q is"),
                     (dict(q=z(T, 64, h).transpose(1, 2)), "must be contiguous"), (dict(c=z(r, T).t()), "must be contiguous"),
                     (dict(norm_weight=z(r, t=F32)), "norm_weight is"), (dict(norm_weight=z(r - 1)), "norm_weight is"),
                     (dict(cache=z(nb, 16, r)), "cache is"), (dict(q=None), "both"), (dict(slot_mapping=i64(1)), "slots for")):
        with pytest.raises(P.PaError, match=match):
            write(**o)
    read = lambda **o: P.pa_latent_read(**{**dict(cache=cache, slot_mapping=i64(T), c=z(T, r), k_rope=z(T, 64), layout=lay), **o})  # noqa: E731
    for o, match in ((dict(c=z(T + 1, r)), "c is"), (dict(k_rope=z(T, 128)[:, :64]), "not contiguous"),
                     (dict(slot_mapping=i64(T).int()), "slot_mapping is")):
        with pytest.raises(P.PaError, match=match):
            read(**o)
    fwd = lambda **o: P.pa_latent_forward(**{**dict(q=z(T, h, r + 64), cache=cache, block_tables=i32(b, 2), seq_lens=i32(b),  # noqa: E731
                                                    query_start_loc=i32(b + 1), max_query_len=2, max_seq_len=32, scale=1.0,
                                                    out=z(T, h, r), workspace=z(64), layout=lay), **o})
    for o, match in ((dict(q=z(T, h, r)), "q is"), (dict(out=z(T, h, r + 64)), "out is"), (dict(block_tables=i32(b + 1, 2)), "block_tables is"),
                     (dict(block_tables=i32(4)), "block_tables is"), (dict(seq_lens=i64(b)), "seq_lens is"),
                     (dict(query_start_loc=i32(b)), "query_start_loc is"), (dict(q=z(T, h, 2 * r + 128)[..., :r + 64]), "not contiguous"),
                     (dict(workspace=z(64, 2)[:, 0]), "workspace is not contiguous")):
        with pytest.raises(P.PaError, match=match):
            fwd(**o)
    assert not launched
    write(), write(q=None, q_out=None), write(norm_weight=z(r)), read(), fwd()
    big = z(T, h, r + 64)
    write(q=z(T, h, 192)[..., 128:], q_out=big[..., r:], c=z(T, r + 64)[:, :r], k_rope=z(T, r + 64)[:, r:])
    assert launched[-1][1] == r + 64 and launched[-1][7:9] == (h * 192, 192) and launched[-1][13:15] == (h * (r + 64), r + 64)


def test_binding_expanded(launched):
    h, d, tk, b = 4, 64, 7, 2
    z = lambda *s, t=BF16: torch.zeros(*s, dtype=t)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    call = lambda **o: P.pa_expanded_forward(**{**dict(q=z(T, h, d + 64), k_nope=z(tk, h, d), k_rope=z(tk, 64), v=z(tk, h, d),  # noqa: E731
                                                       query_start_loc=i32(b + 1), kv_start_loc=i32(b + 1), max_query_len=2,
                                                       max_kv_len=5, scale=1.0, out=z(T, h, d)), **o})
    for o, match in ((dict(q=z(T, h, d)), "q is"), (dict(q=z(T, h, d + 64, t=torch.float16)), "q is"), (dict(v=z(tk, h, d + 8)), "v is"),
                     (dict(k_rope=z(tk + 1, 64)), "k_rope is"), (dict(out=z(T, h * d)), "out is"), (dict(kv_start_loc=i32(b)), "kv_start_loc is"),
                     (dict(query_start_loc=i32(0), kv_start_loc=i32(0)), "empty"), (dict(q=z(T, h * (d + 64))), "q is"),
                     (dict(v=z(tk, d, h).transpose(1, 2)), "must be contiguous"), (dict(query_start_loc=i32(b + 1).long()), "query_start_loc is")):
        with pytest.raises(P.PaError, match=match):
            call(**o)
    assert not launched
    kv = z(tk, h, 2 * d)
    call(), call(k_nope=kv[..., :d], v=kv[..., d:], k_rope=z(tk, 128)[:, 64:])
    lay = launched[-1][-2]
    assert (lay.k_stride, lay.k_head_stride, lay.kr_stride, lay.v_stride, lay.q_head_stride) == (2 * d * h, 2 * d, 128, 2 * d * h, d + 64)
