"""A workspace sized for a step's bounds serves every step within them."""
import itertools

import pytest
import torch

import paged_kv_attention_04_gb300 as P
from latent_cases import Step, check

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
