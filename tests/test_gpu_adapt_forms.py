"""GPU parity of every form of the adapters' kernels (which tile sizes a call
takes follows from its sizes)."""
import pytest
import torch

from few_row_quantized_amd import qgemv as q

from adapt_util import FORMS, adapters, reference, whole_numbers
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


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,n,r,K", [(1, 1, 8, 256), (20, 2, 16, 256), (64, 3, 64, 1024), (64, 1, 128, 512),
                                     (130, 5, 40, 2048), (300, 2, 256, 256), (512, 40, 24, 520)])
def test_sums_of_24_bits_pass_between_the_products(dtype, T, n, r, K):
    """The rank's sums reach the output with all their bits in bf16, within 2^-23
    of the row's largest in fp16 (whole numbers, which the products keep exact)."""
    say(f"adapt, whole numbers {dtype} T={T} n={n} r={r} K={K}")
    *args, v = whole_numbers(T, n, r, K, dtype, seed=T)
    out = q.adapt(*(t.cuda() for t in args)).double().cpu()
    v = v.double()
    if dtype == BF:
        assert torch.equal(out, v)
    else:
        assert ((out - v).abs() <= 2.0 ** -23 * v.amax(1, keepdim=True)).all()
