"""The cache operators' host side at its borders (no GPU): workspaces for calls
of other sizes, streams given by their address, rows too wide to count."""
import pytest
import torch

from few_row_quantized_amd import kv
from few_row_quantized_amd import qgemv as q

from test_host_kv import cache, run_append, run_attend


# ---------------------------------------------------------------- one workspace for smaller calls

def plain_cache(batch, heads, dim, page, width, f8):
    size = 1 if f8 else 2
    scale = 1 << 20 if f8 else None
    return cache(batch=batch, heads=heads, dim=dim, page=page, width=width, stride_head=dim * size,
                 stride_slot=heads * dim * size, stride_page=page * heads * dim * size,
                 dtype=q.E4M3 if f8 else q.BF16, k_scale=scale, v_scale=scale)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,G", [(8, 6), (8, 20), (1, 64), (2, 1), (4, 12)])
def test_a_workspace_is_enough_for_fewer_rows_and_any_window(heads, G, dim, f8):
    """The size for M rows against the calls of up to M: a call is refused where
    it needs more, and with no rows in all nothing is launched.  Batches and
    table widths cross the limits between shared items and items of one
    workgroup, and rows those between one, two and more tiles a wave."""
    L = q.lib()
    row = heads * G * dim
    for batch in (1, 7, 16, 32, 64, 95, 200):
        for width in (2, 8, 13, 63, 125, 126, 2048):
            c = plain_cache(batch, heads, dim, 16, width, f8)
            before = 0
            for M in range(1, q.MAX_M + 1):
                n = L.qgemv_kv_attend_workspace(c, M, heads * G, 0)
                assert n >= before > -1, (batch, width, M)
                before = n
                for m in range(1, M + 1):
                    for window, sinks in ((0, 0), (20, 0), (100, 4), (1900, 64)):
                        assert run_attend(c, xr=row, xh=dim, outr=row, outh=dim, T=0, M=m, heads=heads * G,
                                          window=window, sinks=sinks, nbytes=n) == q.OK, (batch, width, M, m, window)


# ---------------------------------------------------------------- streams by address

def test_the_address_zero_is_the_default_stream(monkeypatch):
    """torch.cuda.ExternalStream(0) makes a stream of torch's pool, which is
    ordered with nothing: it is not what a call on stream 0 runs on."""
    made = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device=None: made.append(s) or ("external", s, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", device))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    on = torch.device("cuda", 0)
    assert kv._allocating(0, on) == ("default", on) and not made
    assert kv._allocating(4096, on) == ("external", 4096, on)
    mine = object()
    assert kv._allocating(mine, on) is mine


# ---------------------------------------------------------------- rows too wide to count

def test_rows_too_wide_for_the_append_are_refused():
    """From 2^26 heads of 256 on, a row's values wrapped and nothing was stored."""
    for heads, dim in ((1 << 26, 256), ((1 << 22) + 1, 256), (1 << 30, 64), ((1 << 31) - 1, 128)):
        c = cache(heads=heads, dim=dim, stride_slot=1 << 45, stride_page=1 << 50, stride_head=dim * 2)
        assert run_append(c, kh=dim, vh=dim, kr=1 << 40, vr=1 << 40) == q.EUNSUPPORTED
        assert run_append(c, kh=dim, vh=dim, kr=1 << 40, vr=1 << 40, T=0) == q.OK
