"""Refusals of the attention over a shared prefix, the rotated append, the routing
and the adapters (no GPU): by the C ABI with fake, never-dereferenced addresses,
and by the Python calls."""
import os
import re

import pytest
import torch

from few_row_quantized_amd import kv
from few_row_quantized_amd import qgemv as q

from test_host_kv import A, BAD_CACHES, HEADER, cache, tensors

FAR = 1 << 40


def run_shared(c, x=A, xr=6144, xh=128, out=A, outr=6144, outh=128, t=q.BF16, lse=None, start=A, n=A, shared=A, T=4,
               M=2, heads=48, window=0, sinks=0, work=A, nbytes=1 << 40):
    return q.lib().qgemv_kv_attend_shared(c, x, xr, xh, out, outr, outh, t, lse, start, n, shared, T, M, heads, window,
                                          sinks, 0.1, work, nbytes, None)


def run_rotated(c, x=A, xr=6144, xh=128, heads=48, out=FAR, outr=6144, outh=128, ot=q.BF16, nk=A, kr=1024, kh=128, nv=A,
                vr=1024, vh=128, src=q.F32, start=A, n=A, T=4, freq=A, pairs=64, position=None, stride=0, axes=0,
                axis=None, interleaved=0):
    return q.lib().qgemv_kv_append_rotated(c, x, xr, xh, heads, out, outr, outh, ot, nk, kr, kh, nv, vr, vh, src, start,
                                           n, T, freq, pairs, position, stride, axes, axis, interleaved, None)


def run_route(x=A, row=256, t=q.F32, bias=None, experts=A, weights=A, T=0, E=256, k=8, score=q.SOFTMAX, groups=1,
              keep=1, best=1, renorm=1):
    return q.lib().qgemv_route(x, row, t, bias, experts, weights, T, E, k, score, groups, keep, best, renorm, 1.0, None)


def run_adapt(y=A, yr=300, out=FAR, outr=300, x=A, xr=512, a=A, b=A, t=q.BF16, adapter=A, scales=None, T=0, n=4, r=16,
              K=512, N=300, work=A, nbytes=1 << 30):
    return q.lib().qgemv_adapt(y, yr, out, outr, x, xr, a, b, t, adapter, scales, T, n, r, K, N, work, nbytes, None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches_refused(kw, want):
    assert run_shared(cache(**kw)) == want
    assert run_rotated(cache(**kw)) == want
    assert q.lib().qgemv_kv_attend_shared_workspace(cache(**kw), 2, 48, 4) == want


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), q.EINVAL), (dict(out=None), q.EINVAL), (dict(start=None), q.EINVAL), (dict(n=None), q.EINVAL),
    (dict(shared=None), q.EINVAL), (dict(T=-1), q.EINVAL), (dict(M=0), q.EINVAL), (dict(M=q.MAX_M + 1), q.EINVAL),
    (dict(heads=0), q.EINVAL), (dict(heads=12), q.EINVAL), (dict(heads=8 * (q.MAX_GROUP + 1)), q.EUNSUPPORTED),
    (dict(t=q.F32), q.EINVAL), (dict(t=q.F16), q.EINVAL), (dict(window=-1), q.EINVAL), (dict(sinks=-1), q.EINVAL),
    (dict(work=None), q.EINVAL), (dict(nbytes=8), q.EINVAL), (dict(xh=64), q.EINVAL), (dict(x=A + 8), q.EALIGN),
    (dict(outr=6148), q.EALIGN), (dict(lse=A + 2), q.EALIGN), (dict(work=A + 8), q.EALIGN),
    (dict(shared=A + 1), q.EALIGN), (dict(T=0), q.OK),
])
def test_attend_shared_refusals(kw, want):
    assert run_shared(cache(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), q.EINVAL), (dict(out=None), q.EINVAL), (dict(nk=None), q.EINVAL), (dict(nv=None), q.EINVAL),
    (dict(start=None), q.EINVAL), (dict(n=None), q.EINVAL), (dict(freq=None), q.EINVAL), (dict(T=-1), q.EINVAL),
    (dict(heads=0), q.EINVAL), (dict(src=q.E4M3), q.EINVAL), (dict(src=9), q.EINVAL), (dict(ot=q.F32), q.EINVAL),
    (dict(ot=q.E4M3), q.EINVAL), (dict(pairs=0), q.EINVAL), (dict(pairs=4), q.EINVAL), (dict(pairs=12), q.EINVAL),
    (dict(pairs=72), q.EINVAL), (dict(pairs=-8), q.EINVAL), (dict(interleaved=2), q.EINVAL),
    (dict(axis=A), q.EINVAL), (dict(position=A), q.EINVAL), (dict(position=A, axes=2, stride=3), q.EINVAL),
    (dict(xh=64), q.EINVAL), (dict(kh=100), q.EINVAL), (dict(vr=64), q.EINVAL), (dict(x=A + 4), q.EALIGN),
    (dict(out=FAR + 8), q.EALIGN), (dict(outr=6148), q.EALIGN), (dict(nk=A + 4), q.EALIGN), (dict(kr=1026), q.EALIGN),
    (dict(start=A + 2), q.EALIGN), (dict(freq=A + 2), q.EALIGN), (dict(position=A + 1, axes=1), q.EALIGN),
    (dict(position=A, axes=1, axis=A + 2), q.EALIGN),
    # over the queries, but not value for value
    (dict(out=A), q.EINVAL), (dict(out=A + 16, src=q.BF16), q.EINVAL), (dict(out=A, src=q.F16), q.EINVAL),
    (dict(out=A, src=q.BF16, outr=6272), q.EINVAL),
    # an output whose rows and heads lie over one another
    (dict(outr=128), q.EINVAL), (dict(outr=6016), q.EINVAL), (dict(outr=256, outh=640), q.EINVAL),
    (dict(out=A, src=q.BF16, outr=128, xr=128), q.EINVAL),
    (dict(T=0), q.OK), (dict(T=0, out=A), q.OK), (dict(T=0, pairs=12), q.EINVAL), (dict(T=1 << 24), q.EUNSUPPORTED),
    (dict(heads=1 << 23, xr=1 << 30, outr=1 << 30, out=1 << 60), q.EUNSUPPORTED),
])
def test_append_rotated_refusals(kw, want):
    assert run_rotated(cache(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), q.EINVAL), (dict(experts=None), q.EINVAL), (dict(weights=None), q.EINVAL), (dict(T=-1), q.EINVAL),
    (dict(t=q.E4M3), q.EINVAL), (dict(t=7), q.EINVAL), (dict(E=0), q.EINVAL), (dict(row=255), q.EINVAL),
    (dict(k=0), q.EINVAL), (dict(k=257), q.EINVAL), (dict(score=2), q.EINVAL), (dict(groups=0), q.EINVAL),
    (dict(groups=3), q.EINVAL), (dict(keep=0), q.EINVAL), (dict(keep=2), q.EINVAL), (dict(best=0), q.EINVAL),
    (dict(best=3), q.EINVAL), (dict(renorm=2), q.EINVAL), (dict(groups=64, keep=1), q.EINVAL),  # 4 experts for 8
    (dict(E=2048, row=2048), q.EUNSUPPORTED), (dict(k=65), q.EUNSUPPORTED),
    (dict(groups=128, keep=64), q.EUNSUPPORTED), (dict(x=A + 2), q.EALIGN), (dict(x=A + 1, t=q.BF16), q.EALIGN),
    (dict(x=A + 2, t=q.BF16), q.OK), (dict(bias=A + 2), q.EALIGN), (dict(experts=A + 2), q.EALIGN),
    (dict(weights=A + 2), q.EALIGN), (dict(), q.OK), (dict(T=1 << 24), q.EUNSUPPORTED),
])
def test_route_refusals(kw, want):
    assert run_route(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(y=None), q.EINVAL), (dict(out=None), q.EINVAL), (dict(x=None), q.EINVAL), (dict(a=None), q.EINVAL),
    (dict(b=None), q.EINVAL), (dict(adapter=None), q.EINVAL), (dict(work=None), q.EINVAL), (dict(T=-1), q.EINVAL),
    (dict(t=q.F32), q.EINVAL), (dict(t=q.E4M3), q.EINVAL), (dict(n=0), q.EINVAL), (dict(r=0), q.EINVAL),
    (dict(r=12), q.EINVAL), (dict(r=264), q.EUNSUPPORTED), (dict(K=0), q.EINVAL), (dict(K=508), q.EINVAL),
    (dict(K=q.MAX_K + 8, xr=q.MAX_K + 8), q.EUNSUPPORTED), (dict(N=0), q.EINVAL), (dict(yr=299), q.EINVAL),
    (dict(outr=299), q.EINVAL), (dict(xr=504), q.EINVAL), (dict(y=A + 2), q.EALIGN), (dict(out=FAR + 1), q.EALIGN),
    (dict(x=A + 8), q.EALIGN), (dict(xr=516), q.EALIGN), (dict(a=A + 4), q.EALIGN), (dict(b=A + 4), q.EALIGN),
    (dict(adapter=A + 2), q.EALIGN), (dict(scales=A + 2), q.EALIGN), (dict(work=A + 4), q.EALIGN),
    (dict(T=4, out=A + 4), q.EINVAL), (dict(T=4, out=A, outr=301), q.EINVAL), (dict(T=4, nbytes=100), q.EINVAL),
    (dict(T=1 << 24, nbytes=1 << 40, out=1 << 60), q.EUNSUPPORTED), (dict(), q.OK), (dict(out=A), q.OK),
])
def test_adapt_refusals(kw, want):
    assert run_adapt(**kw) == want


def test_calls_too_large_for_a_grid_are_refused():
    assert run_shared(cache(batch=1 << 21)) == q.EUNSUPPORTED
    assert run_shared(cache(batch=1 << 14, width=1 << 16)) == q.EUNSUPPORTED
    assert run_shared(cache(width=1 << 16), T=1 << 20) == q.EUNSUPPORTED
    assert run_shared(cache(heads=1), heads=64, T=1 << 25) == q.EUNSUPPORTED


def test_workspace_sizes():
    L = q.lib()
    assert L.qgemv_kv_attend_shared_workspace(cache(), 17, 48, 4) == q.EINVAL
    assert L.qgemv_kv_attend_shared_workspace(cache(), 2, 49, 4) == q.EINVAL
    assert L.qgemv_kv_attend_shared_workspace(cache(), 2, 48, -1) == q.EINVAL
    assert L.qgemv_adapt_workspace(5, 16) > 0 and L.qgemv_adapt_workspace(0, 8) > 0
    assert L.qgemv_adapt_workspace(-1, 16) == q.EINVAL == L.qgemv_adapt_workspace(5, 12) == L.qgemv_adapt_workspace(5, 0)
    assert L.qgemv_adapt_workspace(5, 264) == q.EUNSUPPORTED


@pytest.mark.parametrize("heads,G,dim", [(8, 6, 128), (2, 1, 64), (1, 64, 256), (4, 12, 128)])
def test_a_workspace_is_enough_for_fewer_rows(heads, G, dim):
    """The size for M and T rows against smaller calls: a call is refused where it
    needs more.  Calls here have no rows, or fail at the workspace's size."""
    L = q.lib()
    for batch in (1, 7, 64):
        for width in (1, 2, 63, 2048):
            c = cache(batch=batch, heads=heads, dim=dim, page=16, width=width, stride_head=dim * 2,
                      stride_slot=heads * dim * 2, stride_page=16 * heads * dim * 2)
            for M in (1, 4, 16):
                before = 0
                for T in (0, 1, 21, 22, 43, 128, 500, 2000):
                    n = L.qgemv_kv_attend_shared_workspace(c, M, heads * G, T)
                    assert n >= before > -1
                    before = n
                    row = heads * G * dim
                    for m in range(1, M + 1):
                        for window in (0, 1, 100, 1 << 30):
                            if T == 0:
                                assert run_shared(c, xr=row, outr=row, xh=dim, outh=dim, heads=heads * G, M=m, T=0,
                                                  window=window, nbytes=n) == q.OK
    for T, r in ((1, 8), (511, 256), (512, 8), (513, 16), (5000, 64)):
        n = L.qgemv_adapt_workspace(T, r)
        assert all(L.qgemv_adapt_workspace(t, s) <= n for t in range(0, T + 1, 37) for s in range(8, r + 1, 8))


def test_binding_constants_match_the_header():
    src = open(HEADER).read()
    for name in ("SOFTMAX", "SIGMOID", "MAX_ROUTED", "MAX_GROUPS", "MAX_CHOSEN", "MAX_RANK"):
        assert int(re.search(r"#define\s+QGEMV_%s\s+(\d+)" % name, src).group(1)) == getattr(q, name)


# ---------------------------------------------------------------- Python calls

def test_call_refusals():
    k, v, t = tensors()
    c = q.KvCache(k, v, t)
    start, n = torch.tensor([0, 1, 2, 4], dtype=torch.int32), torch.tensor([3, 4, 5], dtype=torch.int32)
    x, new, one = torch.zeros(4, 6, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 128), torch.zeros(1, dtype=torch.int32)
    x32, freq = x.float(), torch.ones(64)
    at, axes = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(64, dtype=torch.int32)
    logits, bias = torch.zeros(4, 16), torch.zeros(16)
    y, act = torch.zeros(4, 30), torch.zeros(4, 64, dtype=torch.bfloat16)
    a, b = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 30, 8, dtype=torch.bfloat16)
    which, scales = torch.zeros(4, dtype=torch.int32), torch.ones(2)
    for bad in (lambda: q.attend_shared(c, x, start, n, 2, one.long()), lambda: q.attend_shared(c, x, start, n, 2, start),
                lambda: q.attend_shared(c, x.float(), start, n, 2, one),
                lambda: q.attend_shared(c, x, start, n, 2, one, out=x[:3]),
                lambda: q.attend_shared(c, x, start, n, 2, one, lse=torch.zeros(4, 5)),
                lambda: q.attend_shared(c, x, start, n, 2, one, workspace=torch.zeros(1 << 20)),
                lambda: q.attend_shared(c, x, start, n, 2, one),  # not on the GPU
                lambda: q.append_rotated(c, x32, new.half(), new.half(), start, n, freq),
                lambda: q.append_rotated(c, x32.double(), new.double(), new.double(), start, n, freq),
                lambda: q.append_rotated(c, x32[:3], new, new, start, n, freq),
                lambda: q.append_rotated(c, x32[0], new, new, start, n, freq),
                lambda: q.append_rotated(c, x32, new, new[..., :64], start, n, freq),
                lambda: q.append_rotated(c, x32, new, new, start, n, freq.double()),
                lambda: q.append_rotated(c, x32, new, new, start, n, freq[None]),
                lambda: q.append_rotated(c, x32, new, new, start, n, torch.ones(200)),
                lambda: q.append_rotated(c, x32, new, new, start, n, freq, position=at[0]),
                lambda: q.append_rotated(c, x32, new, new, start, n, freq, position=at[:, :3].contiguous()),
                lambda: q.append_rotated(c, x32, new, new, start, n, freq, position=at.long()),
                lambda: q.append_rotated(c, x32, new, new, start, n, freq, axes=axes),
                lambda: q.append_rotated(c, x32, new, new, start, n, freq, position=at, axes=axes[:32]),
                lambda: q.append_rotated(c, x32, new, new, start, n, freq, out=x32),
                lambda: q.append_rotated(c, x32, new, new, start, n, freq, out=x[:3]),
                lambda: q.append_rotated(c, x32, new, new, start, n, freq),  # not on the GPU
                lambda: q.route(logits.double(), 2), lambda: q.route(logits[0], 2), lambda: q.route(logits, 0),
                lambda: q.route(logits, 17), lambda: q.route(logits, 2, score="tanh"),
                lambda: q.route(torch.zeros(4, 32)[:, ::2], 2), lambda: q.route(logits, 2, bias=bias[:3]),
                lambda: q.route(logits, 2, bias=bias.half()), lambda: q.route(logits, 2),  # not on the GPU
                lambda: q.adapt(y.half(), act, a, b, which), lambda: q.adapt(y[0], act, a, b, which),
                lambda: q.adapt(y, act.float(), a, b, which), lambda: q.adapt(y, act[:3], a, b, which),
                lambda: q.adapt(y, act, a.half(), b, which), lambda: q.adapt(y, act, a, b[:1], which),
                lambda: q.adapt(y, act, a[..., :32], b, which), lambda: q.adapt(y, act, a, b.transpose(1, 2), which),
                lambda: q.adapt(y, act, a, b, which.long()), lambda: q.adapt(y, act, a, b, which[:3]),
                lambda: q.adapt(y, act, a, b, which, scales=torch.ones(3)),
                lambda: q.adapt(y, act, a, b, which, out=y[:, :20]), lambda: q.adapt(y.t().contiguous().t(), act, a, b, which),
                lambda: q.adapt(y, act, a, b, which, workspace=torch.zeros(9)),
                lambda: q.adapt(y, act, a, b, which)):  # not on the GPU
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q.attend_shared_workspace(c, 17, 6, 4), lambda: q.adapt_workspace(torch.zeros(2, 9, 64), 4),
                lambda: q.adapt(torch.zeros(4, 30), act, torch.zeros(2, 12, 64, dtype=torch.bfloat16),
                                torch.zeros(2, 30, 12, dtype=torch.bfloat16), which)):
        with pytest.raises(q.QgemvError):
            bad()
    for bad in (lambda: q.attend_shared(c, x, start, n, 2, 64), lambda: q.append_rotated(c, x32, new, new, start, n, None),
                lambda: q.route([1.0], 2), lambda: q.route(logits, "2"), lambda: q.adapt(y, act, a, b, None)):
        with pytest.raises((TypeError, AttributeError)):
            bad()


def test_calls_without_rows():
    k, v, t = tensors()
    c = q.KvCache(k, v, t)
    start, n = torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    x, new = torch.zeros(0, 6, 128), torch.zeros(0, 2, 128)
    one = torch.zeros(1, dtype=torch.int32)
    assert q.attend_shared(c, x.bfloat16(), start, n, 1, one).shape == (0, 6, 128)
    out = q.append_rotated(c, x, new, new, start, n, torch.ones(64))
    assert out.shape == (0, 6, 128) and out.dtype == torch.bfloat16
    e, w = q.route(torch.zeros(0, 16), 3)
    assert e.shape == w.shape == (0, 3) and e.dtype == torch.int32 and w.dtype == torch.float32
    a, b = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 30, 8, dtype=torch.bfloat16)
    assert q.adapt(torch.zeros(0, 30), torch.zeros(0, 64, dtype=torch.bfloat16), a, b,
                   torch.zeros(0, dtype=torch.int32)).shape == (0, 30)


def test_the_calls_are_offered_by_both_modules():
    for name in ("attend_shared", "attend_shared_workspace", "append_rotated", "route", "adapt", "adapt_workspace"):
        assert getattr(q, name) is getattr(kv, name)
