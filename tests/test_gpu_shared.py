"""GPU parity of the attention over a shared prefix against the fp64 oracle of
the attention, at the sizes, masks and layouts where it can go wrong."""
import numpy as np
import pytest
import torch

from few_row_quantized_amd import qgemv as q

from gpu_util import say
from kv_util import KvDevice, KvProblem

pytestmark = pytest.mark.gpu
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
TYPES = [(BF, BF), (HF, HF), (BF, F8), (HF, F8)]


@pytest.fixture(scope="module", autouse=True)
def _gpu(require_gpu):
    torch.cuda.init()
    yield


def problem(shared, rows, lens, poison=True, **kw):
    """A KvProblem whose sequences have the pages of the first `shared` tokens in
    common: those of the first sequence, which has to reach that far."""
    p = KvProblem(rows, lens, **kw)
    pages = min(max(shared, 0) // p.page, p.table.shape[1] - 1)
    p.table[:, :pages] = p.table[0, :pages]
    if poison:
        p.poison()
    return p


def run(d, shared, lse=True, **kw):
    p = d.p
    z = torch.full((p.T, p.H * p.G), float("nan"), device="cuda") if lse is True else lse
    kw.setdefault("scale", p.scale)
    n = torch.tensor([shared], dtype=torch.int32, device="cuda") if isinstance(shared, int) else shared
    out = q.attend_shared(d.cache, kw.pop("q", d.q), d.start, d.len, kw.pop("M", p.M), n, window=p.window,
                          sinks=p.sinks, lse=z, **kw)
    torch.cuda.synchronize()
    return out, z


def parity(p, shared, label, **kw):
    say(f"attend_shared {label}")
    d = KvDevice(p)
    ref = p.reference()
    out, lse = run(d, shared, **kw)
    p.check(out, lse, ref, label)
    return d, ref, out, lse


@pytest.mark.parametrize("qt,ct", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("M,G", [(1, 1), (1, 6), (5, 3), (8, 6), (16, 12)])
def test_shapes(qt, ct, D, M, G):
    rows = [M, max(1, M // 2), M, 1]
    p = problem(130, rows, [240, 131, 128 + M, 300][:4], H=2, G=G, D=D, page=16, q_dtype=qt, dtype=ct, seed=M * G)
    parity(p, 130, f"{qt} {ct} D={D} M={M} G={G}")


@pytest.mark.parametrize("shared", [-5, 0, 1, 15, 16, 31, 32, 33, 63, 64, 65, 127, 128, 192, 400, 10 ** 9])
@pytest.mark.parametrize("qt,ct,D,page", [(BF, BF, 128, 16), (HF, F8, 64, 20), (BF, BF, 256, 1)])
def test_shared_lengths(shared, qt, ct, D, page):
    """Also none, more than a sequence has, and more than the table."""
    p = problem(shared, [3, 2, 1, 4], [420, 300, 5, 200], H=2, G=3, D=D, page=page, q_dtype=qt, dtype=ct, seed=7)
    parity(p, shared, f"shared={shared} {ct} D={D} page={page}")


def test_sequences_that_end_within_the_prefix():
    # before it, at its end, one row on either side, nothing cached, rows before the first token
    p = problem(160, [4, 4, 4, 4, 2, 3, 1], [300, 100, 160, 162, 0, 2, 161], H=2, G=3, D=128, page=16, seed=3)
    _, ref, out, lse = parity(p, 160, "short sequences")
    assert (ref["count"] == 0).sum() == 3


@pytest.mark.parametrize("qt,ct,D", [(BF, BF, 128), (HF, HF, 64), (BF, F8, 128), (HF, F8, 256)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (64, 0), (100, 4), (250, 70), (5000, 2), (40, 10 ** 9)])
def test_windows(qt, ct, D, window, sinks):
    p = problem(200, [3, 5, 1, 2], [460, 205, 330, 150], H=2, G=2, D=D, page=16, q_dtype=qt, dtype=ct, window=window,
                sinks=sinks, seed=window)
    parity(p, 200, f"window={window} sinks={sinks} {ct} D={D}")


def test_more_rows_than_a_tile():
    """Rows of all sequences in tiles of 128, whose borders fall within a row's
    heads; more sequences than threads of a workgroup, some without rows."""
    rows = [(b * 5) % 4 for b in range(300)]
    p = problem(96, rows, [500] + [96 + max(r, 1) + b % 7 for b, r in enumerate(rows)][1:], H=1, G=5, D=64, page=8,
                seed=1)
    parity(p, 96, "300 sequences")
    p = problem(256, [16] * 20, [300 + 3 * b for b in range(20)][::-1], H=2, G=7, D=128, page=32, seed=2)
    parity(p, 256, "2240 rows")


@pytest.mark.parametrize("B,M,H,G,shared,own", [
    (40, 8, 8, 6, 640, 60),    # 120 items: several workgroups for each, each within one
    (60, 8, 8, 6, 448, 600),   # 176: common and own tokens in separate workgroups, and in turn
    (48, 16, 8, 9, 384, 40),   # 432: one for each, or ranges over two
    (64, 16, 8, 12, 128, 30),  # 768: more items than workgroups
])
@pytest.mark.parametrize("ct,D", [(BF, 128), (F8, 64)])
def test_many_items(B, M, H, G, shared, own, ct, D):
    rows = [M if b % 4 else 1 + b % M for b in range(B)]
    lens = [shared + own] + [shared + max(rows[b], own * (b % 5) // 5) for b in range(1, B)]
    p = problem(shared, rows, lens, H=H, G=G, D=D, page=32, dtype=ct, seed=B)
    parity(p, shared, f"{B} sequences of {M} rows, {ct} D={D}")


def test_missing_pages_in_the_prefix():
    p = problem(128, [2, 3, 1], [200, 180, 140], H=2, G=3, D=128, page=16, seed=5, poison=False)
    p.table[:, 2] = -1
    p.table[:, 5] = p.P + 3
    p.poison()
    parity(p, 128, "missing pages")
    p.table[:, :8] = -1  # none of it is there
    p.poison()
    parity(p, 128, "no prefix page")


@pytest.mark.parametrize("qt,ct", TYPES)
def test_values_that_only_some_rows_see(qt, ct):
    """NaNs and infinities in tokens that a window hides from some rows reach
    exactly the rows that see them."""
    p = problem(192, [4, 1, 3], [230, 300, 245], H=2, G=3, D=128, page=16, q_dtype=qt, dtype=ct, window=60, sinks=2,
                seed=8)
    v = p.v.float()
    inf = float("nan") if ct == F8 else float("inf")
    for token, value in ((1, inf), (175, float("nan")), (186, inf), (190, -inf)):
        v[int(p.table[0, token // 16]), token % 16, 1, token % 64] = value
    p.v.copy_(v.to(p.v.dtype))
    d, ref = KvDevice(p), p.reference()
    out, lse = run(d, 192)
    o, want = out.double().cpu().numpy(), ref["out"]
    assert np.isnan(want).any() and np.isfinite(want).any()
    assert np.array_equal(np.isnan(o), np.isnan(want)) and np.array_equal(np.isposinf(o), np.isposinf(want))
    assert np.array_equal(np.isneginf(o), np.isneginf(want))
    finite = np.isfinite(want)
    # the same values without the strays: what is finite has its usual bound
    p2_out = out.clone()
    p2_out[torch.from_numpy(~finite).cuda()] = 0
    for k in ("out", "mass"):
        ref[k][~finite] = 0
    ref["top"] = float(np.nanmax(np.abs(p.v.float().numpy()[np.isfinite(p.v.float().numpy())])))
    p.check(p2_out, lse, ref, "strays")


def test_strided_operands_and_rows_past_the_last_sequence():
    p = problem(64, [2, 3], [150, 90], H=2, G=3, D=64, page=8, seed=4)
    d = KvDevice(p)
    x = torch.randn(p.T + 4, 10, 64, device="cuda").bfloat16()
    x[:p.T, 2:8] = d.q
    out = torch.full((p.T + 4, 8, 64), 7.0, device="cuda", dtype=BF)
    lse = torch.full((p.T + 4, 6), 5.0, device="cuda")
    q.attend_shared(d.cache, x[:, 2:8], d.start, d.len, p.M, torch.tensor([64], dtype=torch.int32, device="cuda"),
                    scale=p.scale, out=out[:, 1:7], lse=lse)
    torch.cuda.synchronize()
    p.check(out[:p.T, 1:7], lse[:p.T], None, "strided")
    assert (out[p.T:] == 7).all() and (out[:, 0] == 7).all() and (out[:, 7] == 7).all() and (lse[p.T:] == 5).all()


def test_head_major_cache_and_rows_past_m():
    p = problem(100, [2, 6], [150, 160], H=4, G=2, D=128, page=20, seed=6)
    k, v = (x.cuda().transpose(1, 2).contiguous().transpose(1, 2) for x in (p.k, p.v))
    d = KvDevice(p)
    d.cache = q.KvCache(k, v, d.table)
    out, lse = run(d, 100)
    p.check(out, lse, None, "head-major")
    fixed = torch.full_like(out, 3.0)
    run(d, 100, out=fixed, M=4)
    assert torch.equal(fixed[:6], out[:6]) and (fixed[6:] == 3).all()


def test_without_lse_and_twice_the_same():
    p = problem(300, [5] * 9, [310 + 17 * b for b in range(9)][::-1], H=3, G=4, D=128, page=16, dtype=F8, seed=9)
    d = KvDevice(p)
    a, _ = run(d, 300)
    b, _ = run(d, 300, lse=None)
    assert torch.equal(a, b)


def test_one_workspace_for_smaller_calls_and_dirty_contents():
    p = problem(128, [8, 3, 8], [300, 180, 250], H=2, G=6, D=128, page=16, seed=10)
    d = KvDevice(p)
    work = q.attend_shared_workspace(d.cache, 16, 12, 4 * p.T)
    work.fill_(0xFF)
    out, lse = run(d, 128, workspace=work)
    p.check(out, lse, None, "dirty workspace")
    again, _ = run(d, 128, workspace=work)
    assert torch.equal(out, again)


def test_captured_and_replayed_with_other_lengths():
    """The prefix, the lengths and the table stay on the device: a captured call
    follows them."""
    p = problem(160, [2, 3, 1], [300, 260, 200], H=2, G=3, D=128, page=16, seed=11)
    d = KvDevice(p)
    shared = torch.tensor([160], dtype=torch.int32, device="cuda")
    work = q.attend_shared_workspace(d.cache, p.M, 6, p.T)
    out, lse = torch.empty_like(d.q), torch.empty((p.T, 6), device="cuda")

    def call():
        q.attend_shared(d.cache, d.q, d.start, d.len, p.M, shared, scale=p.scale, out=out, lse=lse, workspace=work)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n, lens in ((160, [300, 260, 200]), (0, [290, 250, 161]), (48, [170, 260, 60]), (100, [300, 101, 99])):
        shared.fill_(n)
        p.lens, p.len = lens, torch.tensor(lens, dtype=torch.int32)
        d.len.copy_(p.len)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        p.check(out, lse, None, f"replay shared={n}")
        eager, _ = run(d, n)
        assert torch.equal(out, eager)


def test_other_streams():
    p = problem(160, [2, 3, 1], [300, 260, 200], H=2, G=3, D=128, page=16, seed=12)
    d = KvDevice(p)
    want, _ = run(d, 160)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n = torch.tensor([160], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        out = q.attend_shared(d.cache, d.q, d.start, d.len, p.M, n, scale=p.scale, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("qt,ct", [(BF, BF), (HF, F8)])
def test_long_prefix_against_the_attention(qt, ct):
    """Thousands of tokens: against the library's own attention, whose bound
    counts twice (rows of a few heads against the oracle)."""
    B, M, H, G, D, page, shared = 12, 4, 2, 6, 128, 16, 5000
    g = torch.Generator(device="cuda").manual_seed(13)
    lens = [shared + 40 + 97 * b for b in range(B)]
    width = -(-max(lens) // page)
    common = shared // page
    P = common + B * (width - common)
    k, v = ((torch.randn((P, page, H, D), generator=g, device="cuda") * (4 if ct == F8 else 1)).to(ct) for _ in range(2))
    table = torch.empty((B, width), dtype=torch.int32)
    table[:, :common] = torch.arange(common)
    table[:, common:] = common + torch.arange(B * (width - common)).view(B, -1)
    s = torch.full((H,), 0.25, device="cuda") if ct == F8 else None
    cache = q.KvCache(k, v, table.cuda(), s, s)
    start = torch.arange(0, B * M + 1, M, dtype=torch.int32, device="cuda")
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x = (2 * torch.randn((B * M, H * G, D), generator=g, device="cuda")).to(qt)
    la, lb = (torch.empty((B * M, H * G), device="cuda") for _ in range(2))
    a = q.attend(cache, x, start, length, M, lse=la)
    b = q.attend_shared(cache, x, start, length, M, torch.tensor([shared], dtype=torch.int32, device="cuda"), lse=lb)
    torch.cuda.synchronize()
    u = 2.0 ** -8 if qt == BF else 2.0 ** -11
    # each: the weights' rounding (up to u of sum p |v|, here below the largest
    # |v| seen) and the output's own; typical values are far less
    bound = 2 * u * (a.float().abs() + 8.0)
    assert ((a.float() - b.float()).abs() <= bound).all()
    rel = (a.double() - b.double()).norm() / a.double().norm()
    assert rel <= 2 * 2 * u, rel
    assert ((la - lb).abs() <= 1e-4).all()


def test_pages_past_4_gib():
    """Pages anywhere in a large cache give what the same pages close together
    give, and rotated rows go to them."""
    page, H, D, B, width = 64, 8, 128, 3, 7
    g = torch.Generator(device="cuda").manual_seed(1)
    near = [torch.randn(24, page, H, D, device="cuda", generator=g).to(BF) for _ in range(2)]
    far = [torch.empty((1 << 15) + 600, page, H, D, device="cuda", dtype=BF) for _ in range(2)]  # 4.4e9 bytes each
    places = torch.randperm(24, device="cuda", generator=g) * 24 + (1 << 15)
    places[:4] = torch.tensor([0, 9, (1 << 14) + 1, (1 << 15) - 1], device="cuda")
    for a, b in zip(near, far):
        b[places] = a
    table = torch.arange(B * width, device="cuda", dtype=torch.int32).reshape(B, width)
    table[:, :4] = table[0, :4]
    lens, start = torch.tensor([430, 300, 257], dtype=torch.int32, device="cuda"), torch.tensor([0, 4, 7, 8], dtype=torch.int32, device="cuda")
    x = [torch.randn(8, h, D, device="cuda", generator=g) for h in (4 * H, H, H)]
    freq = torch.logspace(0, -4, 64, device="cuda")
    shared = torch.full((1,), 256, dtype=torch.int32, device="cuda")
    results = []
    for (k, v), ids in ((near, table), (far, places[table.long()].int())):
        cache = q.KvCache(k, v, ids)
        turned = q.append_rotated(cache, *x, start, lens, freq)
        lse = torch.empty(8, 4 * H, device="cuda")
        out = q.attend_shared(cache, turned, start, lens, 4, shared, lse=lse)
        results.append((turned, out, lse))
    torch.cuda.synchronize()
    for a, b in zip(*results):
        assert torch.equal(a, b) and torch.isfinite(a.float()).all()
    for a, b in zip(near, far):
        assert torch.equal(a, b[places])
