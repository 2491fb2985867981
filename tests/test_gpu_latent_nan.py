"""A NaN logit reaches the rows that see it, wherever its key stands: first of a request, first of a piece, last."""
import numpy as np
import pytest
import torch

import paged_kv_attention_04_gb300 as P
from latent_cases import Step, check
from test_gpu_expanded import Prompts

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_attention_04_gb300 import build
    build.build()
    P.lib()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keys", [100, 700])
def test_absorbed(keys, dtype):
    """Request r has NaN in the key part alone of its key 16 r (700 keys: cut in three pieces in float32, whose
    borders are at such keys), the last request none."""
    n = -(-keys // 16) + 1
    step = Step(4, 256, [1] * n, [keys] * n, dtype, seed=keys)
    whole = step.want()
    for r in range(n - 1):
        step.cache[step.tables[r, r], 0, 256 + r % 64] = float("nan")
    d = step.run()
    torch.cuda.synchronize()
    assert int(d["status"].item()) == 0
    assert d["out"][:-1].isnan().all()
    check(d["out"][-1:], whole[0][-1:], whole[1][-1:], dtype, step.logit_size(), 320)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shared", [True, False])
def test_expanded(shared, dtype):
    """NaN in the shared key part, or in one head's own, of each request's first, second or last key."""
    step = Prompts(3, 64, [1, 1, 1, 2], [50, 50, 50, 50], dtype, seed=3)
    want, mag = step.want()
    at, size = [0, 51, 149], step.logit_size()
    for k in at:
        if shared:
            step.rope[k, 64 + 7] = float("nan")
        else:
            step.kv[k, 1, 7] = float("nan")
    d = step.run()
    torch.cuda.synchronize()
    assert int(d["status"].item()) == 0
    hit = np.zeros((5, 3), bool)
    hit[:3] = True if shared else np.arange(3) == 1
    assert (d["out"].isnan().all(-1).cpu().numpy() == hit).all()
    check(d["out"][torch.from_numpy(~hit)], want[~hit], mag[~hit], dtype, size, 128)
