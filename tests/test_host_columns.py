"""Operands in columns of one buffer (no GPU): those that overlap are refused."""
import pytest

from few_row_quantized_amd import qgemv as q

from test_host_kv import A, cache
from test_host_step import run_adapt, run_rotated


@pytest.mark.parametrize("at,apart", [
    (300, True), (299, False), (1, False), (-1, False), (-299, False), (-300, True), (700, True), (701, False),
    (-700, True), (-701, False), (1000, False), (1300, True), (-1000, False), (5000, False), (5300, True),
])
def test_adapters_output_beside_the_product(at, apart):
    """y and out, 300 of 1000 columns each, out `at` columns after y: apart, so
    that what is refused is the number of rows, or over one another."""
    y = A + (1 << 20)
    assert (run_adapt(y=y, yr=1000, out=y + 4 * at, outr=1000, T=1 << 24, nbytes=1 << 40)
            == (q.EUNSUPPORTED if apart else q.EINVAL))


def test_adapters_output_in_rows_of_another_length():
    assert run_adapt(y=A, yr=1000, out=A + 4 * 300, outr=1001, T=1 << 24, nbytes=1 << 40) == q.EINVAL


@pytest.mark.parametrize("kw", [
    # 8 of 32 heads of one buffer each, from columns that overlap by a head
    dict(heads=8, x=A, xr=4096, out=A + 7 * 256, outr=4096, src=q.BF16),
    dict(heads=8, x=A + 7 * 256, xr=4096, out=A, outr=4096, src=q.BF16),
    # past the row's end, into the next one's queries
    dict(heads=8, x=A, xr=4096, out=A + 25 * 256, outr=4096, src=q.BF16),
    # heads in turn, which overlap by half
    dict(heads=8, x=A, xr=2048, xh=256, out=A + 128, outr=2048, outh=256, src=q.BF16),
    # heads of other lengths, and rows that do not hold whole ones
    dict(heads=8, x=A, xr=2048, xh=256, out=A + 256, outr=2048, outh=128, src=q.BF16),
    dict(heads=8, x=A, xr=2176, xh=256, out=A + 256, outr=2176, outh=256, src=q.BF16),
    # rows of other lengths in bytes
    dict(heads=8, x=A, xr=4096, out=A + 8 * 512, outr=4096, src=q.F32),
])
def test_rotated_queries_over_the_queries(kw):
    assert run_rotated(cache(), nk=1 << 50, nv=1 << 51, **kw) == q.EINVAL


@pytest.mark.parametrize("kw", [
    dict(out=1 << 41),                                         # where the keys begin
    dict(out=(1 << 41) + 256 * 1024, outr=6144),               # within them
    dict(out=(1 << 42) - 128, outr=6144),                      # over the first value
    dict(heads=8, out=(1 << 41) + 3 * 256, outr=4096, kr=4096, vr=4096, src=q.BF16, nv=(1 << 41) + 8 * 256, x=(1 << 41) + 16 * 256, xr=4096),
])
def test_rotated_queries_over_the_keys_and_values(kw):
    args = dict(nk=1 << 41, nv=1 << 42, T=300)
    args.update(kw)
    assert run_rotated(cache(), **args) == q.EINVAL
