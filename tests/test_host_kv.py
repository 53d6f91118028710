"""Refusals of the cache append, attention and draft acceptance (no GPU): by
the C ABI with fake, never-dereferenced addresses, and by the Python calls."""
import ctypes
import os
import re

import pytest
import torch

from few_row_quantized_amd import qgemv as q

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qgemv.h")
A = 1 << 20


def cache(**kw):
    d = dict(k=A, v=A, table=A, k_scale=None, v_scale=None, stride_page=16 * 8 * 256, stride_slot=8 * 256,
             stride_head=256, pages=10, page=16, width=4, batch=2, heads=8, dim=128, dtype=q.BF16)
    d.update(kw)
    return ctypes.byref(q._KvCacheC(*[d[n] for n, _ in q._KvCacheC._fields_]))


BAD_CACHES = [
    (dict(k=None), q.EINVAL), (dict(v=None), q.EINVAL), (dict(table=None), q.EINVAL),
    (dict(dim=96), q.EINVAL), (dict(dim=0), q.EINVAL), (dict(dtype=q.F32), q.EINVAL), (dict(dtype=7), q.EINVAL),
    (dict(heads=0), q.EINVAL), (dict(pages=0), q.EINVAL), (dict(page=0), q.EINVAL), (dict(width=0), q.EINVAL),
    (dict(batch=0), q.EINVAL), (dict(page=1 << 20, width=1 << 11), q.EINVAL), (dict(stride_slot=0), q.EINVAL),
    (dict(stride_page=-256), q.EINVAL), (dict(dtype=q.E4M3), q.EINVAL), (dict(k_scale=A), q.EINVAL),
    (dict(dtype=q.E4M3, k_scale=A), q.EINVAL), (dict(stride_head=264), q.EALIGN), (dict(k=A + 8), q.EALIGN),
    (dict(table=A + 2), q.EALIGN), (dict(dtype=q.E4M3, k_scale=A + 2, v_scale=A), q.EALIGN),
]


def run_append(c, nk=A, kr=1024, kh=128, nv=A, vr=1024, vh=128, src=q.F32, start=A, n=A, T=4):
    return q.lib().qgemv_kv_append(c, nk, kr, kh, nv, vr, vh, src, start, n, T, None)


def run_attend(c, x=A, xr=6144, xh=128, out=A, outr=6144, outh=128, t=q.BF16, lse=None, start=A, n=A, T=4, M=2,
               heads=48, window=0, sinks=0, work=A, nbytes=1 << 40):
    return q.lib().qgemv_kv_attend(c, x, xr, xh, out, outr, outh, t, lse, start, n, T, M, heads, window, sinks, 0.1,
                                   work, nbytes, None)


def run_verify(p=A, pr=100, d=A, dr=100, t=q.F32, tokens=A, u=A, start=A, out=A, count=A, B=2, T=4, M=2, V=100,
               work=A, nbytes=1 << 40):
    return q.lib().qgemv_verify_drafts(p, pr, d, dr, t, tokens, u, start, out, count, B, T, M, V, work, nbytes, None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches_refused(kw, want):
    assert run_append(cache(**kw)) == want
    assert run_attend(cache(**kw)) == want
    assert q.lib().qgemv_kv_attend_workspace(cache(**kw), 2, 48, 4) == want


def test_null_cache_refused():
    assert run_append(None) == q.EINVAL and run_attend(None) == q.EINVAL


@pytest.mark.parametrize("kw,want", [
    (dict(nk=None), q.EINVAL), (dict(nv=None), q.EINVAL), (dict(start=None), q.EINVAL), (dict(n=None), q.EINVAL),
    (dict(T=-1), q.EINVAL), (dict(src=q.E4M3), q.EINVAL), (dict(src=9), q.EINVAL), (dict(kh=100), q.EINVAL),
    (dict(vr=64), q.EINVAL), (dict(nk=A + 4), q.EALIGN), (dict(kr=1026), q.EALIGN), (dict(start=A + 2), q.EALIGN),
    (dict(T=0), q.OK),
])
def test_append_refusals(kw, want):
    assert run_append(cache(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), q.EINVAL), (dict(out=None), q.EINVAL), (dict(start=None), q.EINVAL), (dict(n=None), q.EINVAL),
    (dict(T=-1), q.EINVAL), (dict(M=0), q.EINVAL), (dict(M=q.MAX_M + 1), q.EINVAL), (dict(heads=0), q.EINVAL),
    (dict(heads=12), q.EINVAL), (dict(heads=8 * (q.MAX_GROUP + 1)), q.EUNSUPPORTED), (dict(t=q.F32), q.EINVAL),
    (dict(t=q.F16), q.EINVAL), (dict(window=-1), q.EINVAL), (dict(sinks=-1), q.EINVAL), (dict(work=None), q.EINVAL),
    (dict(nbytes=8), q.EINVAL), (dict(xh=64), q.EINVAL), (dict(x=A + 8), q.EALIGN), (dict(outr=6148), q.EALIGN),
    (dict(lse=A + 2), q.EALIGN), (dict(work=A + 8), q.EALIGN), (dict(T=0), q.OK),
])
def test_attend_refusals(kw, want):
    assert run_attend(cache(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(p=None), q.EINVAL), (dict(tokens=None), q.EINVAL), (dict(u=None), q.EINVAL), (dict(start=None), q.EINVAL),
    (dict(out=None), q.EINVAL), (dict(count=None), q.EINVAL), (dict(work=None), q.EINVAL), (dict(B=0), q.EINVAL),
    (dict(V=0), q.EINVAL), (dict(T=-1), q.EINVAL), (dict(M=0), q.EINVAL), (dict(M=17), q.EINVAL),
    (dict(t=q.E4M3), q.EINVAL), (dict(pr=99), q.EINVAL), (dict(dr=99), q.EINVAL), (dict(nbytes=0), q.EINVAL),
    (dict(p=A + 2), q.EALIGN), (dict(d=A + 1, t=q.BF16), q.EALIGN), (dict(tokens=A + 2), q.EALIGN),
    (dict(work=A + 4), q.EALIGN),
])
def test_verify_refusals(kw, want):
    assert run_verify(**kw) == want


def test_calls_too_large_for_a_grid_are_refused():
    assert run_append(cache(), T=1 << 24) == q.EUNSUPPORTED
    assert run_verify(B=1 << 24) == q.EUNSUPPORTED
    assert q.lib().qgemv_verify_drafts_workspace(1 << 24, 100) == q.EUNSUPPORTED
    assert run_attend(cache(batch=1 << 21)) == q.EUNSUPPORTED
    assert run_attend(cache(batch=1 << 14, width=1 << 16)) == q.EUNSUPPORTED


def test_workspace_sizes():
    L = q.lib()
    assert L.qgemv_kv_attend_workspace(cache(), 2, 48, 4) > 0
    assert L.qgemv_kv_attend_workspace(cache(), 17, 48, 4) == q.EINVAL
    assert L.qgemv_kv_attend_workspace(cache(), 2, 49, 4) == q.EINVAL
    assert L.qgemv_verify_drafts_workspace(4, 1000) > 0
    assert L.qgemv_verify_drafts_workspace(0, 1000) == q.EINVAL == L.qgemv_verify_drafts_workspace(4, 0)


def test_binding_constants_match_the_header():
    src = open(HEADER).read()
    for name, val in (("QGEMV_F32", q.F32), ("QGEMV_BF16", q.BF16), ("QGEMV_F16", q.F16), ("QGEMV_E4M3", q.E4M3),
                      ("QGEMV_MAX_GROUP", q.MAX_GROUP)):
        assert int(re.search(r"#define\s+%s\s+(\d+)" % name, src).group(1)) == val
    assert "QGEMV_MAX_CONTEXT (1 << 30)" in src and q.MAX_CONTEXT == 1 << 30


# ---------------------------------------------------------------- Python calls

def tensors(D=128, dtype=torch.bfloat16, H=2, P=5, page=4, B=3, width=6):
    return torch.zeros(P, page, H, D, dtype=dtype), torch.zeros(P, page, H, D, dtype=dtype), \
        torch.zeros(B, width, dtype=torch.int32)


def test_cache_construction_refusals():
    k, v, t = tensors()
    q.KvCache(k, v, t)
    q.KvCache(k.transpose(1, 2).contiguous().transpose(1, 2), v.transpose(1, 2).contiguous().transpose(1, 2), t)
    s = torch.ones(2)
    f = torch.float8_e4m3fn
    q.KvCache(k.to(f), v.to(f), t, s, s)
    for bad in (lambda: q.KvCache(k[0], v[0], t), lambda: q.KvCache(k, v[:4], t), lambda: q.KvCache(k, v.half(), t),
                lambda: q.KvCache(k.float(), v.float(), t), lambda: q.KvCache(*tensors(D=96)),
                lambda: q.KvCache(k[:0], v[:0], t), lambda: q.KvCache(k, v, t.long()),
                lambda: q.KvCache(k, v, t[:, ::2]), lambda: q.KvCache(k, v, t[:0]), lambda: q.KvCache(k, v, t, s, s),
                lambda: q.KvCache(k.to(f), v.to(f), t), lambda: q.KvCache(k.to(f), v.to(f), t, s),
                lambda: q.KvCache(k.to(f), v.to(f), t, s, s.double()),
                lambda: q.KvCache(k.to(f), v.to(f), t, s, torch.ones(3)),
                lambda: q.KvCache(torch.zeros(5, 4, 2, 256, dtype=torch.bfloat16)[..., ::2],
                                  torch.zeros(5, 4, 2, 256, dtype=torch.bfloat16)[..., ::2], t),
                lambda: q.KvCache(k, v.transpose(1, 2).contiguous().transpose(1, 2), t)):
        with pytest.raises(ValueError):
            bad()


def test_call_refusals():
    k, v, t = tensors()
    c = q.KvCache(k, v, t)
    start, n = torch.tensor([0, 1, 2, 4], dtype=torch.int32), torch.tensor([3, 4, 5], dtype=torch.int32)
    x, new = torch.zeros(4, 6, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 128)
    prob, tok, u = torch.zeros(4, 9), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    for bad in (lambda: q.append(c, new, new[:3], start, n), lambda: q.append(c, new, new.half(), start, n),
                lambda: q.append(c, new.double(), new.double(), start, n),
                lambda: q.append(c, torch.zeros(4, 3, 128), torch.zeros(4, 3, 128), start, n),
                lambda: q.append(c, new[..., :64], new[..., :64], start, n),
                lambda: q.append(c, new, new, start.long(), n), lambda: q.append(c, new, new, start[:3], n),
                lambda: q.append(c, new, new, start, n[:2]),
                lambda: q.append(c, new, new, start, n),  # not on the GPU
                lambda: q.attend(c, x.float(), start, n, 2), lambda: q.attend(c, x.half(), start, n, 2),
                lambda: q.attend(c, x[..., :64], start, n, 2), lambda: q.attend(c, x[0], start, n, 2),
                lambda: q.attend(c, x, start, n, 2, out=x.half()), lambda: q.attend(c, x, start, n, 2, out=x[:3]),
                lambda: q.attend(c, x, start, n, 2, lse=torch.zeros(4, 5)),
                lambda: q.attend(c, x, start, n, 2, lse=torch.zeros(4, 6).half()),
                lambda: q.attend(c, x, start, n, 2, workspace=torch.zeros(1 << 20)),
                lambda: q.attend(c, x, start, n, 2),  # not on the GPU
                lambda: q.verify(prob.double(), None, tok, u, start, 2),
                lambda: q.verify(prob, prob.half(), tok, u, start, 2), lambda: q.verify(prob, prob[:3], tok, u, start, 2),
                lambda: q.verify(prob, None, tok.long(), u, start, 2), lambda: q.verify(prob, None, tok, u[:3], start, 2),
                lambda: q.verify(prob, None, tok, u, start[:1], 2),
                lambda: q.verify(torch.zeros(4, 18)[:, ::2], None, tok, u, start, 2),
                lambda: q.verify(prob, None, tok, u, start, 2)):  # not on the GPU
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(q.QgemvError):
        q.attend_workspace(c, 17, 6, 4)
    with pytest.raises(q.QgemvError):
        q.attend(c, torch.zeros(4, 5, 128, dtype=torch.bfloat16), start, n, 2)  # 5 query heads on 2


def test_calls_without_rows():
    k, v, t = tensors()
    c = q.KvCache(k, v, t)
    start, n = torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q.append(c, torch.zeros(0, 2, 128), torch.zeros(0, 2, 128), start, n)
    assert q.attend(c, torch.zeros(0, 6, 128, dtype=torch.bfloat16), start, n, 1).shape == (0, 6, 128)
    out, count = q.verify(torch.zeros(0, 9), None, torch.zeros(0, dtype=torch.int32), torch.zeros(0), start, 1)
    assert out.shape == (0,) and count.tolist() == [0, 0, 0]


def test_arguments_of_other_kinds():
    k, v, t = tensors()
    c = q.KvCache(k, v, t)
    start, n = torch.tensor([0, 1, 2, 4], dtype=torch.int32), torch.tensor([3, 4, 5], dtype=torch.int32)
    x, new = torch.zeros(4, 6, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 128)
    for bad in (lambda: q.append(c, [1.0], new, start, n), lambda: q.append(c, new, new, [0, 1, 2, 4], n),
                lambda: q.attend(c, None, start, n, 2), lambda: q.attend(c, x, start, n, "2"),
                lambda: q.attend(c, x, start, n, 2, scale="1"), lambda: q.attend(c, x, start, n, 2, workspace=3),
                lambda: q.verify(None, None, None, None, start, 2)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):
        q.attend(c, x, start, n, 1 << 40)
    with pytest.raises(OverflowError):
        q.attend(c, x, start, n, 2, window=1 << 70)
    with pytest.raises(ValueError):
        q.append(c, torch.zeros(8), torch.zeros(8), start, n)


def test_either_module_can_be_imported_first():
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for first, second in (("kv", "qgemv"), ("qgemv", "kv")):
        code = (f"from few_row_quantized_amd import {first}; from few_row_quantized_amd import {second}; "
                "from few_row_quantized_amd import kv, qgemv; assert qgemv.attend is kv.attend")
        subprocess.run([sys.executable, "-c", code], cwd=root, check=True)
