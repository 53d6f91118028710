"""GPU parity of every form of the adapters' kernels (which tile sizes a call
takes follows from its sizes)."""
import pytest
import torch

from few_row_quantized_amd import qgemv as q

from adapt_util import FORMS, adapters, reference
from gpu_util import say

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu(require_gpu):
    torch.cuda.init()
    yield


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,n,r,K,N", FORMS)
def test_adapt_forms(dtype, T, n, r, K, N):
    say(f"adapt {dtype} T={T} n={n} r={r} K={K} N={N}")
    y, x, a, b, adapter, scales = adapters(T, n, r, K, N, dtype, seed=T + r)
    out = q.adapt(y, x, a, b, adapter, scales=scales)
    torch.cuda.synchronize()
    want, tol = reference(y, x, a, b, adapter, scales)
    bad = ~((out.double() - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}"
    none = adapter < 0
    assert torch.equal(out[none], y[none])
