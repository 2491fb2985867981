"""A workspace sized for a step's bounds serves every step within them."""
import itertools

import pytest
import torch

import paged_kv_attention_04_gb300 as P
from paged_kv_attention_04_gb300 import binding
from latent_cases import Step, check
from test_gpu_expanded import Prompts

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_attention_04_gb300 import build
    build.build()
    P.lib()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads", [1, 8, 9, 40, 256])
@pytest.mark.parametrize("latent", [256, 512])
def test_absorbed_size_never_falls(heads, latent, dtype):
    lay = P.make_latent_layout(heads, latent, 10, dtype)
    size = lambda t, s, q=1: P.pa_latent_workspace_size(lay, min(t, 4), t, q, s)  # noqa: E731
    lens = [1, 16, 255, 256, 257, 4096, 10000, 70000, 1 << 20]
    for s in lens:
        sizes = [size(t, s) for t in itertools.chain(range(1, 700), [1000, 2048, 5000, 40000])]
        assert sizes == sorted(sizes), s
    for t in (1, 3, 100, 607, 608, 3000):
        for q in (1, 2, 7, 40):
            assert [size(t, s, q) for s in lens] == sorted(size(t, s, q) for s in lens)
        assert [size(t, 4096, q) for q in (1, 2, 7, 40)] == sorted(size(t, 4096, q) for q in (1, 2, 7, 40))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_absorbed_steps_within_the_bounds(dtype):
    """One workspace, sized for 1000 tokens, for steps of 1 to 620; what lies behind it stays as it was."""
    heads, latent, most = 8, 256, 3000
    lay = P.make_latent_layout(heads, latent, 10, dtype)
    n = P.pa_latent_workspace_size(lay, 1000, 1000, 8, most)
    room = torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    for lens in ([most], [300, 2999, 1], [50 + i for i in range(100)], [1 + i % 90 for i in range(620)]):
        step = Step(heads, latent, [1] * len(lens), lens, dtype, seed=len(lens))
        d = step.gpu()
        d["ws"] = room[:n]
        step.run(d, max_q=1)
        torch.cuda.synchronize()
        assert int(d["status"].item()) == 0 and (room[n:] == 0x5a).all()
        want, mag = step.want()
        check(d["out"], want, mag, dtype, step.logit_size(), latent + 64)


def test_expanded_size_of_one_token_is_the_largest():
    size = P.pa_expanded_workspace_size
    for heads, head_size in ((1, 64), (32, 128), (256, 128)):
        for n in (1000, 1024, 8192, 100000):
            assert max(size(heads, head_size, t, n) for t in range(1, 50000, 777)) <= size(heads, head_size, 1, n)
        sizes = [size(heads, head_size, 1, n) for n in (1, 1000, 1024, 8192, 1 << 20)]
        assert size(heads, head_size, 1, binding._CUT_KEYS - 1) == 0 < size(heads, head_size, 1, binding._CUT_KEYS)
        assert sizes == sorted(sizes)


def expanded_call(step, d, ws, nbytes):
    """The C call, with a workspace as it is given."""
    lay = P.pa_expanded_layout(step.heads, step.size, 64, P.PA_BF16, d["q"].stride(0), d["q"].stride(1), d["k"].stride(0),
                               d["k"].stride(1), d["kr"].stride(0), d["v"].stride(0), d["v"].stride(1))
    return P.lib().pa_expanded_forward(d["q"].data_ptr(), d["k"].data_ptr(), d["kr"].data_ptr(), d["v"].data_ptr(),
                                       d["qsl"].data_ptr(), d["kvsl"].data_ptr(), len(step.q_lens), step.tokens, step.keys,
                                       int(step.q_lens.max()), int(step.seq_lens.max()), step.scale, d["out"].data_ptr(), ws,
                                       nbytes, lay, d["status"].data_ptr(), torch.cuda.current_stream().cuda_stream)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are none")
def test_expanded_takes_an_empty_workspace():
    """A size of 0 for a large step, in an arena's address: a smaller step takes it as none."""
    lay = P.pa_expanded_layout(4, 128, 64, P.PA_BF16, 768, 192, 1024, 256, 64, 1024, 256)
    assert P.pa_expanded_workspace_size(4, 128, 100, 4096) > 0
    rc = P.lib().pa_expanded_forward(256, 256, 256, 256, 256, 256, 2, 100, 4096, 100, 4096, 0.1, 256, 256, 0, lay, None, None)
    assert rc == P.PA_ERR_CUDA  # (past every check of arguments: there is no device)


@pytest.mark.gpu
def test_expanded_empty_workspace_is_none():
    step = Prompts(4, 128, [300, 20], [3000, 1500], seed=5)
    d = step.gpu()
    room = torch.full((4096,), 0x5a, dtype=torch.uint8, device="cuda")
    assert expanded_call(step, d, None, 0) == P.PA_OK
    torch.cuda.synchronize()
    first = d["out"].clone()
    step.check(d)
    d["out"].fill_(7.0)
    assert expanded_call(step, d, room.data_ptr(), 0) == P.PA_OK
    torch.cuda.synchronize()
    assert torch.equal(d["out"], first) and (room == 0x5a).all() and int(d["status"].item()) == 0
