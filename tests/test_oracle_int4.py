"""Pins of the 4-bit cache's oracle (format, rounding, corner cases) and the host
checks of the calls that take a 4-bit cache."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import int4
import paged_kv_attention_04_gb300 as P


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_04_gb300 import build
    build.build()
    return P.lib()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("is_v", [False, True])
def test_a_page_is_filled_exactly(D, is_v):
    """Every code has a nibble of its own and every parameter two bytes; together
    they are the page."""
    byte, nib, par = int4._maps(is_v, D)
    taken = set(zip(byte.ravel().tolist(), nib.ravel().tolist()))
    assert len(taken) == 16 * D
    at = np.concatenate([par.ravel(), par.ravel() + 1]).tolist()
    assert sorted(at + [b for b, n in taken if n == 0]) == list(range(10 * D))
    assert (par % 2 == 0).all()


@pytest.mark.parametrize("is_v", [False, True])
def test_round_trip_is_within_half_a_step(is_v):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 16, 2, 64)).astype(np.float32)
    got = int4.dequantise(int4.pack(x, 0.5, is_v), 0.5, is_v)
    step = np.repeat(int4.params(int4.pack(x, 0.5, is_v), is_v)[0].astype(np.float64), 32, -1) * 0.5
    # half a step, and what clamping code 15 and rounding z in f16 add: 15 s off by
    # 2^-11 of the range (15 steps), z by 2^-11 of |z| (below 4 / 0.5 here, 8)
    assert (np.abs(got - x) <= step * (0.5 + 15 * 2.0 ** -11) + 8 * 0.5 * 2.0 ** -11).all()


def test_store_is_pack_row_by_row():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((2, 16, 2, 64)).astype(np.float32)
    for is_v in (False, True):
        empty = np.full((2, 2, 640), 0xA5, np.uint8)
        got = int4.store(empty, x.reshape(32, 2, 64)[::-1], np.arange(32)[::-1], 1.0, is_v)
        assert np.array_equal(got, int4.pack(x, 1.0, is_v))
        assert np.array_equal(int4.store(empty, x[0], np.full(16, -1), 1.0, is_v), empty)


def test_quantiser_corner_cases():
    x = np.zeros((6, 32), np.float32)
    x[0] = 3.0                       # equal values: s = 0
    x[1, 5] = np.nan
    x[2, :2] = np.inf, -np.inf       # saturate
    x[3] = np.arange(32) / 2.0       # s = 15.5 / 15
    x[4, :16] = 15.0                 # s = 1, values on the grid
    x[5, 0], x[5, 1], x[5, 2] = 30.0, 1.0, 3.0   # s = 2: 1 and 3 are ties -> codes 0 and 2
    c, s, z = int4.quantise(x, 1.0)
    assert s[0, 0] == 0 and z[0, 0] == 3 and not c[0].any()
    assert np.isnan(s[1, 0]) and np.isnan(z[1, 0]) and not c[1].any()
    assert z[2, 0] == -16384 and c[2, 0] == 15 and c[2, 1] == 0 and np.isfinite(s[2, 0])
    assert c[3, 0] == 0 and c[3, 31] == 15
    assert s[4, 0] == 1 and c[4, 0] == 15 and c[4, 31] == 0
    assert s[5, 0] == 2 and c[5, 0] == 15 and c[5, 1] == 0 and c[5, 2] == 2
    # the largest range keeps every value, and z - 16 s, finite in f16
    assert abs(float(z[2, 0]) - 16 * float(s[2, 0])) < 65504


def L(**kw):
    base = dict(num_q_heads=32, num_kv_heads=8, head_size=128, num_blocks=100, dtype=torch.bfloat16,
                cache_dtype=P.PA_INT4)
    base.update(kw)
    return P.make_layout(**base)


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=torch.float32), P.PA_ERR_UNSUPPORTED),
    (dict(head_size=96), P.PA_ERR_UNSUPPORTED),
    (dict(block_size=32), P.PA_ERR_UNSUPPORTED),
    (dict(k_scale=0.0), P.PA_ERR_INVALID),
    (dict(v_scale=float("nan")), P.PA_ERR_INVALID),
    (dict(v_scale=-1.0), P.PA_ERR_INVALID),
    (dict(cache_dtype=4), P.PA_ERR_INVALID),
])
def test_bad_layouts_are_refused(lib, bad, code):
    lay = L(**bad)
    assert lib.pa_forward_workspace_size(ctypes.byref(lay), 4, 4, 64) == 0
    for call in (lib.pa_cache_write, lib.pa_cache_read):
        assert call(16, 16, 16, 1, 16, 16, ctypes.byref(lay), None, None) == code
        assert P.last_error()


def test_cache_read_argument_checks(lib):
    for lay in (L(), L(cache_dtype=None), L(cache_dtype=P.PA_FP8_E4M3)):
        def read(kc=16, vc=16, slots=16, n=3, k=16, v=16, status=None):
            return lib.pa_cache_read(kc, vc, slots, n, k, v, ctypes.byref(lay), status, None)
        assert read(None, None, None, 0, None, None) == P.PA_OK
        for bad in (dict(kc=None), dict(vc=None), dict(slots=None), dict(k=None), dict(v=None), dict(n=-1),
                    dict(kc=24), dict(vc=8), dict(k=24), dict(v=4), dict(slots=20), dict(status=2)):
            assert read(**bad) == P.PA_ERR_INVALID, bad
    assert lib.pa_cache_read(16, 16, 16, 1, 16, 16, None, None, None) == P.PA_ERR_INVALID


def test_layout_of_a_4_bit_cache():
    lay = P.layout_of(torch.zeros(7, 2, 640, dtype=torch.uint8), 8, k_scale=0.5, v_scale=2.0)
    assert (lay.head_size, lay.num_kv_heads, lay.num_blocks, lay.block_size) == (64, 2, 7, 16)
    assert (lay.dtype, lay.cache_dtype, lay.k_scale, lay.v_scale) == (P.PA_BF16, P.PA_INT4, 0.5, 2.0)
    assert P.cache_shape(lay) == (7, 2, 640)
    assert P.cache_shape(L(cache_dtype=None)) == (100, 16, 8, 128)
    with pytest.raises(P.PaError, match="page"):
        P.layout_of(torch.zeros(7, 2, 641, dtype=torch.uint8), 8)


def test_binding_rejects_host_tensors():
    kc = torch.zeros(4, 2, 640, dtype=torch.uint8)
    e = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(P.PaError, match="not a CUDA tensor"):
        P.pa_cache_read(kc, kc, torch.zeros(1, dtype=torch.int64), e, e, P.layout_of(kc, 8))
