"""The rotated append's angles over the whole range that the header names."""
import numpy as np
import pytest
import torch

import oracle
from few_row_quantized_amd import qgemv as q

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu(require_gpu):
    torch.cuda.init()
    yield


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("low,high", [(1e-5, 1.0), (0.5, 1.0), (1.0, 500.0)])
def test_far_positions_by_any_frequency(low, high, interleaved):
    """Pairs of 1 and 0, which turn into cosine and sine: within 2^-22 and half a
    step of fp16, at positions of all 32 bits, while the angle is below 2^40."""
    say(f"turns of frequencies {low}..{high} interleaved={interleaved}")
    g = torch.Generator().manual_seed(int(high))
    T, D, pairs = 64, 128, 64
    position = torch.randint(-2 ** 31, 2 ** 31, (1, T), generator=g, dtype=torch.int64)
    position[0, :6] = torch.tensor([-2 ** 31, 2 ** 31 - 1, 0, -1, 2 ** 30, 2 ** 24 + 1])
    freq = (low * (high / low) ** torch.rand(pairs, generator=g)).float()
    x = torch.zeros(T, 1, D)
    if interleaved:
        x[..., 0::2] = 1.0
    else:
        x[..., :pairs] = 1.0
    k, v = (torch.zeros(4, 16, 1, D, dtype=torch.float16, device="cuda") for _ in range(2))
    cache = q.KvCache(k, v, torch.arange(4, dtype=torch.int32, device="cuda")[None].contiguous())
    start, length = (torch.tensor(n, dtype=torch.int32, device="cuda") for n in ([0, T], [T]))
    out = q.append_rotated(cache, x.cuda(), x.cuda(), x.cuda(), start, length, freq.cuda(),
                           position=position.int().cuda(), interleaved=interleaved)
    torch.cuda.synchronize()
    want = oracle.rotate_reference(x.double().numpy(), position.tolist(), freq.double().numpy(), None, interleaved)
    for name, got in (("queries", out), ("keys", k.view(T, 1, D))):
        off = np.abs(got.double().cpu().numpy() - want)
        tol = 2.0 ** -22 + np.maximum(2.0 ** -11 * np.abs(want), 2.0 ** -25)
        assert (off <= tol).all(), f"{name}: {(off > tol).sum()} of {off.size}, worst {(off / tol).max():.3g} of the tolerance"
