"""What the slot write and the read-back refuse before a kernel could run out of bounds, and
what they pass on.  The device check and the launch are replaced, so nothing runs on a GPU."""
import pytest
import torch

import paged_kv_attention_04_gb300 as P
from paged_kv_attention_04_gb300 import binding

NB, H, D, T = 4, 2, 64, 3


@pytest.fixture
def launched(monkeypatch):
    calls = []
    monkeypatch.setattr(binding, "lib", lambda: type("L", (), dict(pa_cache_write="write", pa_cache_read="read")))
    monkeypatch.setattr(binding, "_on_one_device", lambda **tensors: 0)
    monkeypatch.setattr(binding, "_launch", lambda fn, dev, stream, *args: calls.append((fn, args)))
    return calls


def call(kind="write", dtype=torch.bfloat16, cache=None, **over):
    lay = P.make_layout(4 * H, H, D, NB, dtype, cache_dtype=cache)
    kc = torch.zeros(P.cache_shape(lay), dtype=dtype if cache is None else torch.uint8)
    a = dict(k=torch.zeros(T, H, D, dtype=dtype), v=torch.zeros(T, H, D, dtype=dtype),
             slots=torch.zeros(T, dtype=torch.int64))
    a.update(over)
    if kind == "write":
        P.pa_cache_write(a["k"], a["v"], a["slots"], kc, kc.clone(), lay)
    else:
        P.pa_cache_read(kc, kc.clone(), a["slots"], a["k"], a["v"], lay)


CACHES = [(torch.bfloat16, None), (torch.float32, None), (torch.bfloat16, P.PA_FP8_E4M3), (torch.bfloat16, P.PA_INT4)]


@pytest.mark.parametrize("kind", ["write", "read"])
@pytest.mark.parametrize("dtype,cache", CACHES)
def test_refusals(launched, kind, dtype, cache):
    wide = torch.float64 if dtype == torch.float32 else torch.float32
    row = lambda n, h=H, t=dtype: torch.zeros(n, h, D, dtype=t)  # noqa: E731
    for over, match in ((dict(slots=torch.zeros(2 * T, dtype=torch.int32)), "slot_mapping"),
                        (dict(slots=torch.zeros(T - 1, dtype=torch.int64)), "slots for|rows"),
                        (dict(v=row(T - 1)), "v is"), (dict(v=row(T, 1)), "v is"), (dict(k=row(T, 1)), "k is"),
                        (dict(k=row(T, t=wide)), "k is"), (dict(v=row(T, t=wide)), "v is"),
                        (dict(k=row(T, t=torch.uint8)), "k is")):
        with pytest.raises(P.PaError, match=match):
            call(kind, dtype, cache, **over)
    assert not launched


@pytest.mark.parametrize("dtype,cache", CACHES)
def test_what_is_in_bounds_passes(launched, dtype, cache):
    call("write", dtype, cache)
    call("write", dtype, cache, k=torch.zeros(T, H * D, dtype=dtype), v=torch.zeros(T + 2, H, D, dtype=dtype),
         slots=torch.zeros(T + 4, dtype=torch.int64))
    call("write", dtype, cache, k=torch.zeros(0, H, D, dtype=dtype))
    call("read", dtype, cache)
    assert [fn for fn, _ in launched] == ["write"] * 3 + ["read"]
    assert [a[3] for fn, a in launched] == [T, T, 0, T]


@pytest.mark.parametrize("dtype,bits", [(torch.bfloat16, torch.int16), (torch.float32, torch.int32)])
def test_unquantised_rows_may_come_as_bits(launched, dtype, bits):
    call("write", dtype, None, k=torch.zeros(T, H, D, dtype=bits), v=torch.zeros(T, H, D, dtype=bits))
    assert len(launched) == 1
    if dtype == torch.bfloat16:
        for cache in (P.PA_FP8_E4M3, P.PA_INT4):
            with pytest.raises(P.PaError, match="k is"):
                call("write", dtype, cache, k=torch.zeros(T, H, D, dtype=bits))
