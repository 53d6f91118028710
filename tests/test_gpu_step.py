"""GPU parity of the rotated append, the routing to experts and the adapters
against the fp64 oracle, at the sizes, masks and layouts where they can go wrong."""
import numpy as np
import pytest
import torch

import oracle
from few_row_quantized_amd import qgemv as q

from gpu_util import say
from kv_util import STEP, KvDevice, KvProblem
from test_gpu_kv import append_expected, same_bits

pytestmark = pytest.mark.gpu
F32, BF, HF, F8 = torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu(require_gpu):
    torch.cuda.init()
    yield


# ---------------------------------------------------------------- rotated append

def frequencies(pairs, base=10000.0):
    return (base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float()


def places(p):
    at = torch.zeros(p.T, dtype=torch.int32)
    for t, b, pos in oracle.kv_oracle.row_places(p.start.tolist(), p.lens):
        at[t] = pos
    return at


def rounding(t, value, scale=1.0):
    """Half a step of type t at value / scale, in units of value."""
    x = np.abs(value) / scale
    if t == F8:
        return np.maximum(2.0 ** -4 * x, 2.0 ** -10) * scale
    if t == HF:
        return np.maximum(2.0 ** -11 * x, 2.0 ** -25)
    return 2.0 ** -8 * x


def near(got, want, before, t, scale, label):
    """got within want's rounding to t, and within the rotation's own error before
    it: cos and sin off by 2^-22, two products and a sum in fp32 (3 roundings of at
    most |a| + |b|), for E4M3 the division."""
    sizes = np.abs(before)  # |a| + |b| of the pair, or nothing where it is not turned
    off = sizes * (2.0 ** -22 + 3 * 2.0 ** -24) + 2.0 ** -23 * np.abs(want) * (t == F8)
    tol = off + rounding(t, np.abs(want) + off, scale)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{label}: {bad.sum()} of {bad.size}, first {tuple(np.argwhere(bad)[0])}: "
                           f"{got[bad][0]} for {want[bad][0]}, tolerance {np.broadcast_to(tol, bad.shape)[bad][0]}")


def pair_sizes(x, pairs, interleaved):
    """|a| + |b| of the pair of each value, 0 past the pairs."""
    s = np.zeros(x.shape)
    a = np.abs(x)
    if interleaved:
        both = a[..., 0:2 * pairs:2] + a[..., 1:2 * pairs:2]
        s[..., 0:2 * pairs:2] = s[..., 1:2 * pairs:2] = both
    else:
        s[..., :pairs] = s[..., pairs:2 * pairs] = a[..., :pairs] + a[..., pairs:2 * pairs]
    return s


def check_rotated(p, d, x, new_k, new_v, freq, position, axes, interleaved, out, label):
    """The queries, the cache's rotated rows, and all else bit for bit."""
    at = places(p)[None] if position is None else position
    pairs = len(freq)
    args = (at.tolist(), freq.double().numpy(), None if axes is None else axes.tolist(), interleaved)
    rows = [t for t, _, _ in oracle.kv_oracle.row_places(p.start.tolist(), p.lens)]
    f = x.double().numpy()
    want = oracle.rotate_reference(f, *args)
    near(out.double().cpu().numpy()[rows], want[rows], pair_sizes(f, pairs, interleaved)[rows], out.dtype, 1.0, label + " q")
    f = new_k.double().numpy()
    want, sizes = oracle.rotate_reference(f, *args), pair_sizes(f, pairs, interleaved)
    plain_k, plain_v = append_expected(p, new_k, new_v)
    assert same_bits(d.v, plain_v), label
    got = d.k.clone()
    if 2 * pairs < p.D:
        assert same_bits(got[..., 2 * pairs:], plain_k[..., 2 * pairs:]), label
    for t, i, s in oracle.append_places(p.table.numpy(), p.start.tolist(), p.lens, p.page, p.P):
        scale = np.ones((p.H, 1)) if p.k_scale is None else p.k_scale.double().numpy()[:, None]
        value = got[i, s].double().cpu().numpy() * scale
        w = np.clip(want[t], -448 * scale, 448 * scale) if p.k_scale is not None else want[t]
        n = 2 * pairs
        near(value[:, :n], w[:, :n], sizes[t][:, :n], p.dtype, scale, label + " k")
        got[i, s] = plain_k[i, s].to(got.device)
    assert same_bits(got, plain_k), f"{label}: slots of no row"


@pytest.mark.parametrize("src", [F32, BF, HF])
@pytest.mark.parametrize("dtype", [BF, HF, F8])
@pytest.mark.parametrize("D,H,G,page,pairs,interleaved", [
    (64, 1, 1, 1, 32, False), (64, 2, 3, 7, 8, True), (128, 8, 6, 16, 64, False), (128, 3, 2, 16, 40, False),
    (128, 2, 4, 16, 64, True), (256, 5, 1, 20, 128, False), (256, 2, 2, 20, 24, True), (256, 1, 12, 20, 120, False)])
def test_append_rotated(src, dtype, D, H, G, page, pairs, interleaved):
    label = f"{src} -> {dtype} D={D} pairs={pairs} {'interleaved' if interleaved else 'halves'}"
    say(f"append_rotated {label}")
    # a row before the first position, a sequence without rows, positions that cross pages
    p = KvProblem([3, 0, 16, 1, 2], [40, 7, 16, 33, 1], H=H, G=G, D=D, page=page, q_dtype=HF if dtype == HF else BF,
                  dtype=dtype)
    g = torch.Generator().manual_seed(9)
    x = torch.randn((p.T, H * G, D), generator=g).to(src)
    new_k, new_v = ((10.0 * torch.randn((p.T, H, D), generator=g)).to(src) for _ in range(2))
    d, freq = KvDevice(p), frequencies(pairs)
    out = q.append_rotated(d.cache, x.cuda(), new_k.cuda(), new_v.cuda(), d.start, d.len, freq.cuda(),
                           interleaved=interleaved)
    torch.cuda.synchronize()
    assert out.dtype == (HF if dtype == HF else BF)
    check_rotated(p, d, x, new_k, new_v, freq, None, None, interleaved, out, label)


@pytest.mark.parametrize("A,interleaved", [(1, False), (3, False), (3, True), (5, True)])
def test_given_positions_on_several_axes(A, interleaved):
    p = KvProblem([3, 5, 1], [40, 300, 33], H=2, G=3, D=128, page=16, dtype=BF)
    g = torch.Generator().manual_seed(A)
    x = torch.randn((p.T, 6, 128), generator=g)
    new_k, new_v = (torch.randn((p.T, 2, 128), generator=g) for _ in range(2))
    position = torch.randint(-50, 1 << 21, (A, p.T), generator=g, dtype=torch.int32)
    axes = torch.randint(0, A, (48,), generator=g, dtype=torch.int32) if A > 1 else None
    if A == 5:
        axes[3], axes[4] = -7, 90  # limited to the axes that are there
    d, freq = KvDevice(p), frequencies(48)
    out = torch.empty((p.T, 6, 128), dtype=HF, device="cuda")
    got = q.append_rotated(d.cache, x.cuda(), new_k.cuda(), new_v.cuda(), d.start, d.len, freq.cuda(),
                           position=position.cuda(), axes=None if axes is None else axes.cuda(),
                           interleaved=interleaved, out=out)
    torch.cuda.synchronize()
    assert got is out
    check_rotated(p, d, x, new_k, new_v, freq, position, axes, interleaved, out, f"{A} axes")


def test_rotation_in_place_and_from_one_product():
    """Columns of one product, whose queries are turned where they are."""
    p = KvProblem([2, 5], [9, 30], H=4, G=2, D=128, page=8, dtype=BF)
    qkv = torch.randn(p.T, 16, 128).bfloat16()
    for interleaved in (False, True):
        d, freq, x = KvDevice(p), frequencies(64), qkv.cuda()
        out = q.append_rotated(d.cache, x[:, :8], x[:, 8:12], x[:, 12:], d.start, d.len, freq.cuda(),
                               interleaved=interleaved, out=x[:, :8])
        torch.cuda.synchronize()
        check_rotated(p, d, qkv[:, :8], qkv[:, 8:12], qkv[:, 12:], freq, None, None, interleaved, out, "in place")
        assert torch.equal(x[:, 8:].cpu(), qkv[:, 8:])


def test_rotation_drops_rows_without_a_page_and_leaves_rows_of_no_sequence():
    p = KvProblem([4, 4, 2], [20, 8, 50], H=2, G=2, D=64, page=4, dtype=BF)
    p.table[0, 4] = -1                       # positions 16..19: not there
    p.table[1, 1] = p.P                      # an id past the pages
    p.lens[2] = (p.table.shape[1]) * 4 + 1   # its last row lies past the table
    p.len[2] = p.lens[2]
    p.table[2, -1] = 1
    x = torch.randn(p.T + 3, 4, 64)
    new = torch.randn(p.T + 3, 2, 64)
    d, freq = KvDevice(p), frequencies(32)
    out = torch.full((p.T + 3, 4, 64), 7.0, dtype=BF, device="cuda")
    q.append_rotated(d.cache, x.cuda(), new.cuda(), -new.cuda(), d.start, d.len, freq.cuda(), out=out)
    torch.cuda.synchronize()
    assert (out[p.T:] == 7).all()
    check_rotated(p, d, x[:p.T], new[:p.T], -new[:p.T], freq, None, None, False, out[:p.T], "dropped rows")


def test_rotation_of_nan_and_infinite_values():
    p = KvProblem([2], [9], H=1, G=1, D=64, page=8, dtype=BF)
    x, new = torch.randn(2, 1, 64), torch.randn(2, 1, 64)
    x[0, 0, 3], x[1, 0, 5], x[1, 0, 60] = float("nan"), float("inf"), float("nan")
    d, freq = KvDevice(p), frequencies(16)
    out = q.append_rotated(d.cache, x.cuda(), new.cuda(), new.cuda(), d.start, d.len, freq.cuda()).float().cpu()
    # a pair takes its partner with it, a value past the pairs nothing
    assert out[0, 0].isnan().nonzero().flatten().tolist() == [3, 19]
    assert set((~out[1, 0].isfinite()).nonzero().flatten().tolist()) == {5, 21, 60}


def test_rotation_captured_and_replayed():
    p = KvProblem([2, 3], [20, 40], H=2, G=2, D=64, page=8, dtype=BF)
    d, freq = KvDevice(p), frequencies(32).cuda()
    x, new = torch.randn(p.T, 4, 64, device="cuda"), torch.randn(p.T, 2, 64, device="cuda")
    out = torch.empty((p.T, 4, 64), dtype=BF, device="cuda")
    fresh_k, fresh_v = d.k.clone(), d.v.clone()
    q.append_rotated(d.cache, x, new, -new, d.start, d.len, freq, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.append_rotated(d.cache, x, new, -new, d.start, d.len, freq, out=out)
    for lens in ([20, 40], [11, 3], [21, 36]):
        d.k.copy_(fresh_k)
        d.v.copy_(fresh_v)
        p.lens, p.len = lens, torch.tensor(lens, dtype=torch.int32)
        d.len.copy_(p.len)
        graph.replay()
        torch.cuda.synchronize()
        check_rotated(p, d, x.cpu(), new.cpu(), -new.cpu(), freq.cpu(), None, None, False, out, f"replay {lens}")


# ---------------------------------------------------------------- routing

def check_route(x, k, experts, weights, label, **kw):
    ref = dict(kw)
    ref["softmax"] = ref.pop("score", "softmax") == "softmax"
    if ref.get("bias") is not None:
        ref["bias"] = ref["bias"].double().numpy()
    e, w = oracle.route_reference(x.double().numpy(), k, **ref)
    got = experts.cpu().numpy()
    assert np.array_equal(got, e), f"{label}: rows {np.argwhere((got != e).any(1))[:5].ravel()}"
    # one rounding to fp32 of a value that fp64 gives to some 10^-15
    z = weights.double().cpu().numpy()
    assert (np.abs(z - w) <= (2.0 ** -24 + 1e-12) * np.abs(w) + 2.0 ** -149).all(), label


ROUTES = [dict(), dict(score="sigmoid"), dict(renormalise=False, scale=2.5), dict(bias=True),
          dict(score="sigmoid", bias=True, scale=2.5), dict(score="sigmoid", renormalise=False)]


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (5, 63, 6), (4, 64, 64), (7, 65, 8), (300, 128, 8), (33, 160, 6),
                                   (9, 257, 4), (260, 512, 22), (2, 1000, 64), (2, 1024, 1)])
@pytest.mark.parametrize("kw", ROUTES)
def test_route(dtype, T, E, k, kw):
    g = torch.Generator().manual_seed(E + k)
    x = (2 * torch.randn((T, E), generator=g)).to(dtype)
    kw = dict(kw)
    if kw.get("bias"):
        kw["bias"] = 0.1 * torch.randn(E, generator=g)
    dev = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    experts, weights = q.route(x.cuda(), k, **dev)
    torch.cuda.synchronize()
    check_route(x, k, experts, weights, f"{dtype} T={T} E={E} k={k} {kw}", **kw)


@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score,bias", [("sigmoid", True), ("softmax", False), ("softmax", True)])
@pytest.mark.parametrize("E,groups,keep,k", [(256, 8, 4, 8), (160, 8, 3, 6), (60, 4, 2, 9), (64, 64, 8, 8), (63, 7, 1, 9),
                                             (96, 3, 3, 10), (1024, 16, 5, 12), (8, 2, 1, 1)])
def test_route_by_groups(E, groups, keep, k, score, bias, best):
    g = torch.Generator().manual_seed(E)
    x = torch.randn((70, E), generator=g).bfloat16()
    kw = dict(score=score, groups=groups, keep=keep, best=best, bias=0.1 * torch.randn(E, generator=g) if bias else None)
    dev = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    experts, weights = q.route(x.cuda(), k, **dev)
    torch.cuda.synchronize()
    check_route(x, k, experts, weights, f"E={E} groups={groups}", **kw)


def test_route_equal_choices_go_by_number():
    x = torch.zeros(3, 200)
    x[1, ::2] = 1.0
    x[2] = torch.arange(200) % 3
    for kw in (dict(), dict(score="sigmoid"), dict(bias=torch.zeros(200)), dict(groups=4, keep=2, best=2)):
        dev = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
        experts, weights = q.route(x.cuda(), 10, **dev)
        check_route(x, 10, experts, weights, str(kw), **kw)


def test_route_of_experts_that_are_not_there():
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(3)
    x = torch.randn((12, 40), generator=g)
    x[torch.rand((12, 40), generator=g) < 0.6] = -inf
    x[2] = -inf
    x[3] = nan
    x[4, 1:] = -inf
    x[5, ::2] = nan
    x[6] = torch.finfo(F32).min
    x[7, 3] = torch.finfo(F32).max
    x[8] = -800.0  # whose sigmoids are 0 in fp64
    bias = 0.1 * torch.randn(40, generator=g)
    bias[5], bias[6] = -inf, nan
    for kw in (dict(), dict(score="sigmoid"), dict(bias=bias), dict(score="sigmoid", bias=bias, groups=5, keep=2, best=2),
               dict(groups=8, keep=2), dict(renormalise=False, groups=4, keep=4, best=2)):
        dev = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
        experts, weights = q.route(x.cuda(), 6, **dev)
        torch.cuda.synchronize()
        check_route(x, 6, experts, weights, str({k: v for k, v in kw.items() if k != "bias"}), **kw)


def test_route_strided_rows_and_a_side_stream():
    x = torch.randn(50, 300).cuda()
    want = q.route(x[:, 100:228].contiguous(), 8)
    got = q.route(x[:, 100:228], 8)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        got = q.route(x[:, 100:228], 8, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_route_feeds_the_gathered_product():
    """Rows through their experts: routing, the gathered 4-bit product, the sum
    by weights; experts that are not there are skipped."""
    from few_row_quantized_amd import synth
    s = synth.MoeShape("route_moe", 12, 512, 256, 4, 64, 4, (4,), 9)
    m = synth.make_moe_problem(s)
    T, k = 4, 4
    logits = torch.randn(T, 12, generator=torch.Generator().manual_seed(1))
    logits[3, 2:] = float("-inf")
    experts, weights = q.route(logits.cuda(), k)
    x_idx = torch.arange(T, dtype=torch.int32).repeat_interleave(k).cuda()
    y = torch.zeros((T * k, s.N), device="cuda")
    q.qgemv_gather(torch.from_numpy(m.codes).cuda(), torch.from_numpy(m.scales.view(np.int16)).cuda(),
                   torch.from_numpy(m.biases.view(np.int16)).cuda(), torch.from_numpy(m.x.view(np.int16)).cuda(), x_idx,
                   experts, y, T * k, T, s.E, s.N, s.K, s.bits, s.group_size)
    out = (y.view(T, k, s.N) * weights[..., None]).sum(1).double().cpu().numpy()
    e, w = oracle.route_reference(logits.double().numpy(), k)
    pairs = [(t, j) for t in range(T) for j in range(k) if e[t, j] >= 0]
    xi, ei = np.array([t for t, _ in pairs], np.int32), np.array([e[t, j] for t, j in pairs], np.int32)
    args = (m.codes, m.scales, m.biases, m.x, xi, ei, s.N, s.K, s.bits, s.group_size)
    ref, size = oracle.qgemv_gather_reference(*args), oracle.gather_abs_product_sum(*args)
    want, tol = np.zeros((T, s.N)), np.zeros((T, s.N))
    for i, (t, j) in enumerate(pairs):
        want[t] += w[t, j] * ref[i]
        tol[t] += w[t, j] * (1e-3 * size[i] + 1e-6)
    assert len(pairs) == 14 and (np.abs(out - want) <= 1.001 * tol).all()


# ---------------------------------------------------------------- adapters

def adapters(T, n, r, K, N, dtype=BF, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    y, x = torch.randn((T, N), generator=g), torch.randn((T, K), generator=g).to(dtype)
    a = (torch.randn((n, r, K), generator=g) * (spread * K ** -0.5)).to(dtype)
    b = (torch.randn((n, N, r), generator=g) * r ** -0.5).to(dtype)
    return y, x, a, b, torch.randint(-1, n, (T,), generator=g, dtype=torch.int32), 0.5 + torch.rand(n, generator=g)


def check_adapt(out, y, x, a, b, adapter, scales, label):
    """The bound: K products summed in fp32 in parts of any order, K + 8 roundings;
    the sums in parts (2^-24 of each in bf16; in fp16 2^-23 of the row's largest,
    with 2^-17 kept here for both and the sum over the rank); r products of the
    parts; scale and the sum with y, 3 roundings."""
    d = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    ref, down, up = oracle.adapt_reference(d(y), d(x), d(a), d(b), adapter.tolist(), d(scales))
    K, r = x.shape[1], a.shape[1]
    tol = ((K + 8) * 2.0 ** -24 * down + (2.0 ** -17 + (2 * r + 8) * 2.0 ** -24) * up
           + 3 * 2.0 ** -24 * (np.abs(d(y)) + np.abs(ref)))
    o = out.double().cpu().numpy()
    bad = ~(np.abs(o - ref) <= tol)
    assert not bad.any(), f"{label}: {bad.sum()} of {bad.size}, first {tuple(np.argwhere(bad)[0])}: {o[bad][0]} for {ref[bad][0]}"


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,n,r,K,N", [
    (1, 1, 8, 64, 16), (5, 8, 16, 512, 96), (16, 1, 16, 256, 130), (17, 1, 32, 264, 64), (40, 1, 64, 320, 50),
    (70, 1, 8, 136, 33), (64, 64, 8, 128, 40), (65, 3, 24, 1000, 77), (77, 5, 8, 1000, 251), (200, 4, 128, 256, 100),
    (130, 90, 16, 128, 64), (512, 2, 16, 64, 48), (513, 3, 40, 72, 20), (1100, 5, 16, 64, 17), (3, 2, 256, 2048, 300),
    (90, 1, 256, 96, 65), (2, 300, 16, 8, 1)])
def test_adapt(dtype, T, n, r, K, N):
    say(f"adapt {dtype} T={T} n={n} r={r} K={K} N={N}")
    y, x, a, b, adapter, scales = adapters(T, n, r, K, N, dtype, seed=T + r)
    out = q.adapt(y.cuda(), x.cuda(), a.cuda(), b.cuda(), adapter.cuda(), scales=scales.cuda())
    torch.cuda.synchronize()
    check_adapt(out, y, x, a, b, adapter, scales, f"{dtype} T={T} n={n} r={r} K={K} N={N}")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,n,r,K,N", [
    (512, 8, 16, 256, 16000), (64, 1, 72, 64, 44000), (64, 1, 200, 40, 44000),  # tiles of 64 rows
    (64, 2, 72, 64, 27000), (512, 16, 40, 64, 10500), (200, 8, 16, 64, 20000),  # of 32
    (512, 300, 24, 64, 40), (100, 500, 8, 64, 20), (512, 256, 48, 128, 30),  # many adapters
    (300, 40, 256, 512, 70), (5, 8, 128, 4096, 64)])  # several tiles of ranks a wave, and one
def test_adapt_tiles(dtype, T, n, r, K, N):
    say(f"adapt {dtype} T={T} n={n} r={r} K={K} N={N}")
    y, x, a, b, adapter, scales = adapters(T, n, r, K, N, dtype, seed=T + r)
    out = q.adapt(y.cuda(), x.cuda(), a.cuda(), b.cuda(), adapter.cuda(), scales=scales.cuda())
    torch.cuda.synchronize()
    check_adapt(out, y, x, a, b, adapter, scales, f"{dtype} T={T} n={n} r={r} K={K} N={N}")


def test_adapt_in_place_columns_and_rows_without_an_adapter():
    """Columns of a wider product, in place; rows without an adapter, of any
    number outside, keep their bits."""
    y, x, a, b, adapter, scales = adapters(30, 4, 16, 128, 70, seed=1)
    adapter[3], adapter[4], adapter[5] = -1, 4, -2 ** 31
    wide, rows = torch.randn(30, 200), torch.randn(30, 304).bfloat16()
    wide[:, 33:103], rows[:, 96:224] = y, x
    w, xs = wide.cuda(), rows.cuda()
    view = w[:, 33:103]
    with pytest.raises(q.QgemvError):  # rows of x 300 values apart are not 16-byte aligned
        q.adapt(view, torch.zeros(30, 300, device="cuda", dtype=BF)[:, 96:224], a.cuda(), b.cuda(), adapter.cuda(), out=view)
    assert q.adapt(view, xs[:, 96:224], a.cuda(), b.cuda(), adapter.cuda(), out=view) is view
    torch.cuda.synchronize()
    check_adapt(view, y, x, a, b, adapter, None, "in place")
    assert torch.equal(w[:, :33].cpu(), wide[:, :33]) and torch.equal(w[:, 103:].cpu(), wide[:, 103:])
    assert torch.equal(view[3:6].cpu(), y[3:6])


def test_adapt_without_any_adapter_copies():
    y, x, a, b, adapter, scales = adapters(70, 4, 16, 128, 70, seed=2)
    adapter.fill_(-1)
    out = q.adapt(y.cuda(), x.cuda(), a.cuda(), b.cuda(), adapter.cuda())
    assert torch.equal(out.cpu(), y)


def test_adapt_rows_do_not_depend_on_others():
    y, x, a, b, adapter, scales = adapters(40, 3, 16, 256, 64, seed=3)
    adapter[:] = torch.arange(40) % 3
    args = [t.cuda() for t in (y, x, a, b, adapter)]
    want = q.adapt(*args)
    again = q.adapt(*args)
    assert torch.equal(want, again)
    x2, y2 = args[1].clone(), args[0].clone()
    x2[7], y2[11] = float("nan"), float("inf")
    got = q.adapt(y2, x2, *args[2:])
    torch.cuda.synchronize()
    keep = [t for t in range(40) if t not in (7, 11)]
    assert torch.equal(got[keep], want[keep]) and got[7].isnan().all() and got[11].isinf().all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("spread", [1e-4, 3e3])
def test_adapt_small_and_large_sums(dtype, spread):
    """Sums between the two products past fp16's range above, and where it loses
    bits below."""
    y, x, a, b, adapter, scales = adapters(20, 2, 32, 512, 64, dtype, seed=4, spread=spread)
    x = (x.float() * 30).to(dtype)
    out = q.adapt(y.cuda(), x.cuda(), a.cuda(), b.cuda(), adapter.cuda(), scales=scales.cuda())
    torch.cuda.synchronize()
    check_adapt(out, y, x, a, b, adapter, scales, f"spread={spread}")


def test_adapt_captured_dirty_workspace_and_streams():
    y, x, a, b, adapter, scales = adapters(48, 6, 16, 512, 200, seed=5)
    y, x, a, b, at, scales = (t.cuda() for t in (y, x, a, b, adapter, scales))
    want = q.adapt(y, x, a, b, at, scales=scales)
    work = q.adapt_workspace(a, 600)
    work.fill_(0xFF)
    out = torch.empty_like(y)
    q.adapt(y, x, a, b, at, scales=scales, out=out, workspace=work)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.adapt(y, x, a, b, at, scales=scales, out=out, workspace=work)
    for shift in (1, 2, 5):
        at.copy_((adapter.cuda() + shift) % 7 - 1)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, q.adapt(y, x, a, b, at, scales=scales))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        got = q.adapt(y, x, a, b, at, scales=scales, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, got)
