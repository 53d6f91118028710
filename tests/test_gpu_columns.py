"""Outputs in other columns of their input's buffer."""
import pytest
import torch

from few_row_quantized_amd import qgemv as q

from adapt_util import adapters, reference
from kv_util import KvDevice, KvProblem
from test_gpu_step import check_rotated, frequencies

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu(require_gpu):
    torch.cuda.init()
    yield


@pytest.mark.parametrize("T,N,gap,first", [(30, 70, 0, False), (30, 70, 5, True), (90, 33, 0, True)])
def test_adapted_rows_beside_the_product(T, N, gap, first):
    y, x, a, b, adapter, scales = adapters(T, 4, 16, 128, N, BF, seed=T)
    wide = torch.full((T, 2 * N + gap), 5.0, device="cuda")
    left, right = wide[:, :N], wide[:, N + gap:]
    src, out = (right, left) if first else (left, right)
    src.copy_(y)
    assert q.adapt(src, x, a, b, adapter, scales=scales, out=out) is out
    torch.cuda.synchronize()
    want, tol = reference(y, x, a, b, adapter, scales)
    assert ((out.double() - want).abs() <= tol).all() and torch.equal(src, y)
    assert (wide[:, N:N + gap] == 5).all()
    at = gap + 1 if first else N - 1  # so that they have one column in common
    with pytest.raises(q.QgemvError):
        q.adapt(src, x, a, b, adapter, out=wide[:, at:at + N])


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("parts", [3, 4])
def test_rotated_queries_of_heads_side_by_side(parts, heads_first):
    """A head's query, key and value one after another: turned in place, or to a
    place of their own after them."""
    p = KvProblem([2, 5], [9, 30], H=4, G=1, D=64, page=8, dtype=BF)
    rows = torch.randn(p.T, 4, parts, 64, generator=torch.Generator().manual_seed(2)).bfloat16()
    d, freq, x = KvDevice(p), frequencies(32), rows.cuda()
    if heads_first:
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
    out = q.append_rotated(d.cache, x[:, :, 0], x[:, :, 1], x[:, :, 2], d.start, d.len, freq.cuda(),
                           out=x[:, :, 0 if parts == 3 else 3])
    torch.cuda.synchronize()
    check_rotated(p, d, rows[:, :, 0], rows[:, :, 1], rows[:, :, 2], freq, None, None, False, out, "side by side")
    assert torch.equal(x[:, :, 1:3].cpu(), rows[:, :, 1:3])
    with pytest.raises(q.QgemvError):
        q.append_rotated(d.cache, x[:, :, 0], x[:, :, 1], x[:, :, 2], d.start, d.len, freq.cuda(), out=x[:, :, 1])


@pytest.mark.parametrize("src", [BF, torch.float16])
def test_rotated_queries_beside_the_queries(src):
    """Queries, keys, values and the turned queries in one buffer."""
    p = KvProblem([2, 5], [9, 30], H=4, G=2, D=128, page=8, dtype=src, q_dtype=src)
    rows = torch.randn(p.T, 24, 128, generator=torch.Generator().manual_seed(1)).to(src)
    d, freq, x = KvDevice(p), frequencies(64), rows.cuda()
    out = q.append_rotated(d.cache, x[:, :8], x[:, 8:12], x[:, 12:16], d.start, d.len, freq.cuda(), out=x[:, 16:])
    torch.cuda.synchronize()
    check_rotated(p, d, rows[:, :8], rows[:, 8:12], rows[:, 12:16], freq, None, None, False, out, "beside")
    assert torch.equal(x[:, :16].cpu(), rows[:, :16])
    with pytest.raises(q.QgemvError):
        q.append_rotated(d.cache, x[:, :8], x[:, 8:12], x[:, 12:16], d.start, d.len, freq.cuda(), out=x[:, 1:9])
