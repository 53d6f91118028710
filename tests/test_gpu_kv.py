"""GPU parity of the cache append, the attention over the cache and the draft
acceptance against the fp64 oracle, at the sizes, masks and layouts where they
can go wrong."""
import numpy as np
import pytest
import torch

import oracle
from few_row_quantized_amd import qgemv as q

from gpu_util import say
from kv_util import KvDevice, KvProblem, draft_problem

pytestmark = pytest.mark.gpu
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu(require_gpu):
    torch.cuda.init()
    yield


# ---------------------------------------------------------------- append

def bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16)


def append_expected(p, new_k, new_v):
    """The cache after the append, in the cache's type, on the CPU: torch's own
    casts (round to nearest even), after the division and the limit for 8 bits."""
    k, v = p.k.clone(), p.v.clone()
    for x, new, scale in ((k, new_k, p.k_scale), (v, new_v, p.v_scale)):
        y = new.float()
        if scale is not None:
            y = y / scale[None, :, None]
            y = torch.where(y > 448, 448.0, torch.where(y < -448, -448.0, y))
        y = y.to(x.dtype)
        for t, i, s in oracle.append_places(p.table.numpy(), p.start.tolist(), p.lens, p.page, p.P):
            x[i, s] = y[t]
    return k, v


def same_bits(a, b):
    """Equal bit for bit, NaNs apart, whose payload is free."""
    a, b = a.cpu(), b.cpu()
    both = a.float().isnan() & b.float().isnan()
    return bool((both | (bits(a) == bits(b))).all())


@pytest.mark.parametrize("src", [torch.float32, BF, HF])
@pytest.mark.parametrize("dtype", [BF, HF, F8])
@pytest.mark.parametrize("D,H,page", [(64, 1, 1), (128, 8, 16), (256, 5, 20)])
def test_append(src, dtype, D, H, page):
    say(f"append {src} -> {dtype} D={D} H={H} page={page}")
    # a row before the first position, a sequence without rows, positions that cross pages
    p = KvProblem([3, 0, 16, 1, 2], [40, 7, 16, 33, 1], H=H, D=D, page=page, q_dtype=HF if dtype == HF else BF, dtype=dtype)
    g = torch.Generator().manual_seed(9)
    new_k, new_v = ((300.0 * torch.randn((p.T, H, D), generator=g)).to(src) for _ in range(2))
    new_k[0, 0, :6] = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-9]).to(src)
    want_k, want_v = append_expected(p, new_k, new_v)
    d = KvDevice(p)
    q.append(d.cache, new_k.cuda(), new_v.cuda(), d.start, d.len)
    torch.cuda.synchronize()
    assert same_bits(d.k, want_k) and same_bits(d.v, want_v)


def test_append_strided_sources_and_head_major_cache():
    p = KvProblem([2, 5], [9, 30], H=4, D=128, page=8, dtype=BF)
    qkv = torch.randn(p.T, 16, 128)  # queries, keys and values of one product
    want_k, want_v = append_expected(p, qkv[:, 8:12], qkv[:, 12:])
    k, v = (x.cuda().transpose(1, 2).contiguous().transpose(1, 2) for x in (p.k, p.v))
    x = qkv.cuda()
    q.append(q.KvCache(k, v, p.table.cuda()), x[:, 8:12], x[:, 12:], p.start.cuda(), p.len.cuda())
    torch.cuda.synchronize()
    assert same_bits(k, want_k) and same_bits(v, want_v)
    # keys and values in one allocation [pages, 2, page, heads, dim]
    kv = torch.stack([p.k, p.v], 1).cuda()
    q.append(q.KvCache(kv[:, 0], kv[:, 1], p.table.cuda()), x[:, 8:12], x[:, 12:], p.start.cuda(), p.len.cuda())
    torch.cuda.synchronize()
    assert same_bits(kv[:, 0], want_k) and same_bits(kv[:, 1], want_v)


def test_append_drops_rows_without_a_page():
    p = KvProblem([4, 4, 2], [20, 8, 50], H=2, D=64, page=4, dtype=BF)
    p.table[0, 4] = -1                       # positions 16..19: not there
    p.table[1, 1] = p.P                      # an id past the pages
    p.lens[2] = (p.table.shape[1]) * 4 + 1   # its last row lies past the table
    p.len[2] = p.lens[2]
    p.table[2, -1] = 1
    new = torch.randn(p.T, 2, 64)
    want_k, want_v = append_expected(p, new, -new)
    d = KvDevice(p)
    q.append(d.cache, new.cuda(), -new.cuda(), d.start, d.len)
    torch.cuda.synchronize()
    assert same_bits(d.k, want_k) and same_bits(d.v, want_v)


def test_append_many_sequences():
    # more sequences than threads of a workgroup, some without rows
    rows = [(b * 7) % 3 for b in range(700)]
    p = KvProblem(rows, [max(r, 1) + b % 5 for b, r in enumerate(rows)], H=1, D=64, page=2, dtype=BF)
    new = torch.randn(p.T, 1, 64)
    want_k, want_v = append_expected(p, new, -new)
    d = KvDevice(p)
    q.append(d.cache, new.cuda(), -new.cuda(), d.start, d.len)
    torch.cuda.synchronize()
    assert same_bits(d.k, want_k) and same_bits(d.v, want_v)


# ---------------------------------------------------------------- attend

TYPES = [(BF, BF), (HF, HF), (BF, F8), (HF, F8)]


def parity(p, label, **kw):
    say(f"attend {label}")
    d = KvDevice(p)
    ref = p.reference()
    out, lse = d.attend(**kw)
    p.check(out, lse, ref, label)
    return d, ref, out, lse


@pytest.mark.parametrize("qt,ct", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("M,G", [(1, 1), (1, 6), (5, 3), (3, 12), (8, 6), (16, 4), (16, 12)])
def test_attend_shapes(qt, ct, D, M, G):
    rows = [M, max(1, M // 2), M, 1]
    p = KvProblem(rows, [130, 75, M, 300], H=2, G=G, D=D, page=16, q_dtype=qt, dtype=ct, seed=M * G, poison=True)
    parity(p, f"{qt} {ct} D={D} M={M} G={G}")


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257, 511, 1025])
@pytest.mark.parametrize("qt,ct,D,page", [(BF, BF, 128, 16), (HF, F8, 64, 20), (BF, BF, 256, 1)])
def test_attend_lengths(n, qt, ct, D, page):
    p = KvProblem([1, min(n, 3)], [n, n], H=2, G=3, D=D, page=page, q_dtype=qt, dtype=ct, seed=n, poison=True)
    parity(p, f"n={n} {ct} D={D} page={page}")


@pytest.mark.parametrize("page", [1, 2, 3, 7, 8, 20, 33, 64, 100, 128, 1000])
def test_attend_pages(page):
    p = KvProblem([4, 2], [391, 128], H=1, G=5, D=128, page=page, seed=page, poison=True)
    parity(p, f"page={page}")


@pytest.mark.parametrize("window", [1, 2, 16, 31, 32, 33, 100, 250, 5000])
@pytest.mark.parametrize("sinks", [0, 1, 4, 33, 64, 400])
def test_attend_windows(window, sinks):
    p = KvProblem([7, 1, 16], [389, 100, 16], H=2, G=2, D=64, page=16, q_dtype=HF, window=window, sinks=sinks,
                  seed=window + sinks, poison=True)
    parity(p, f"window={window} sinks={sinks}")


def test_attend_long_window_over_long_context():
    p = KvProblem([5, 3, 1], [9000, 5003, 4100], H=2, G=4, D=64, page=64, q_dtype=HF, window=4096, sinks=4, poison=True)
    parity(p, "window 4096 of 9000")


@pytest.mark.parametrize("ct", [BF, F8])
def test_attend_split_over_a_long_context(ct):
    p = KvProblem([5], [20001], H=2, G=6, D=128, page=16, dtype=ct, poison=True)
    parity(p, f"one sequence of 20001 {ct}")


@pytest.mark.parametrize("M,G,seqs,n", [(5, 10, 7, 7900), (2, 2, 9, 9400), (5, 16, 9, 9400), (3, 48, 7, 7900)])
def test_attend_long_ranges(M, G, seqs, n):
    """Enough tokens that the workgroups of a CU take unequal shares: two and
    three of them, with rows in one wave and over four."""
    lens = [n + 97 * b - 41 * b * b for b in range(seqs)]
    p = KvProblem([M] * (seqs - 1) + [1], lens, H=8, G=G, D=64, page=64, seed=n + G)
    parity(p, f"{seqs} sequences of {n}, {M * G} rows")


@pytest.mark.parametrize("B,M,G,n", [(60, 1, 2, 1000), (70, 2, 10, 2000), (50, 5, 16, 1000)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5)])
def test_attend_items_of_one_workgroup_each(B, M, G, n, window, sinks):
    """Items of up to 32 and 64 tiles that no two workgroups share, the table as
    wide as the longest; one sequence with no token, one with fewer than rows."""
    lens = [n - (37 * b * b) % (n - 20) for b in range(B - 2)] + [0, 1]
    p = KvProblem([1 + b % M for b in range(B)], lens, H=4, G=G, D=64, page=8, window=window, sinks=sinks, seed=n + G,
                  extra_width=0)
    parity(p, f"{B} sequences, {M * G} rows")


@pytest.mark.parametrize("ct", [BF, F8])
@pytest.mark.parametrize("lens", [[16, 31, 32, 33, 97, 128], [129, 20, 64], [5000, 300]])
def test_attend_64_rows(ct, lens):
    p = KvProblem([16] * (len(lens) - 1) + [13], lens, H=3, G=4, D=128, page=16, dtype=ct, seed=sum(lens), poison=True,
                  extra_width=0)
    parity(p, f"64 rows, {lens} {ct}")


def test_attend_ragged_batch():
    g = np.random.default_rng(4)
    lens = [int(x) for x in np.exp(g.uniform(0, np.log(3000), 37))]
    p = KvProblem([min(n, 1 + b % 4) for b, n in enumerate(lens)], lens, H=3, G=2, D=64, page=16, seed=4, poison=True)
    parity(p, "37 sequences")


def test_attend_many_short_sequences():
    # more sequences than threads of a workgroup, some without rows, some without tokens
    rows = [b % 3 for b in range(600)]
    lens = [0 if b % 11 == 0 else (b * 13) % 70 for b in range(600)]
    p = KvProblem(rows, lens, H=1, G=2, D=64, page=8, seed=6)
    parity(p, "600 sequences")


@pytest.mark.parametrize("window", [0, 3])
def test_rows_that_see_nothing(window):
    # nothing cached; fewer tokens than rows (the first rows lie before the first token)
    p = KvProblem([3, 4, 2], [0, 2, 40], H=2, G=3, D=128, page=16, window=window, poison=True)
    d, ref, out, lse = parity(p, "empty rows")
    assert (out[:5] == 0).all() and torch.isneginf(lse[:5]).all() and torch.isfinite(lse[5:]).all()


def test_pages_that_are_not_there_are_not_seen():
    p = KvProblem([2, 3, 1], [300, 95, 60], H=2, G=2, D=128, page=16, window=0)
    p.table[0, 3] = -1
    p.table[0, 4] = p.P
    p.table[1, 5] = 2 ** 31 - 1
    p.table[2, :] = -7  # nothing left
    p.poison()
    d, ref, out, lse = parity(p, "missing pages")
    assert torch.isneginf(lse[5]).all() and (out[5] == 0).all()


def test_length_past_the_table_counts_as_the_tables():
    p = KvProblem([2], [64], H=1, G=2, D=64, page=16, extra_width=0)
    d = KvDevice(p)
    want, _ = d.attend()
    d.len = torch.tensor([10 ** 9], dtype=torch.int32, device="cuda")
    got, _ = d.attend()
    assert torch.equal(want, got)


def test_starts_outside_the_rows_are_limited():
    p = KvProblem([2, 2], [40, 50], H=1, G=2, D=64, page=16)
    d = KvDevice(p)
    want, _ = d.attend()
    d.start = torch.tensor([-5, 2, 900], dtype=torch.int32, device="cuda")
    out = torch.full_like(d.q, 7.0)
    d.attend(out=out, M=16)  # no access out of range; sequence 1's rows are not its own any more
    d.start = torch.tensor([3, 2, 1], dtype=torch.int32, device="cuda")
    out = torch.full_like(d.q, 7.0)
    d.attend(out=out)
    assert (out == 7.0).all()


def test_rows_past_m_are_left_alone():
    p = KvProblem([6], [90], H=1, G=2, D=64, page=16)
    d = KvDevice(p)
    want, _ = d.attend()
    out = torch.full_like(d.q, 7.0)
    d.attend(out=out, M=4)
    assert (out[4:] == 7.0).all()
    p.check(torch.cat([out[:4], want[4:]]), None)


@pytest.mark.parametrize("qt,ct", TYPES)
def test_what_unseen_slots_hold_does_not_matter_within_a_tile(qt, ct):
    """A draft row's own key and value are NaN or infinite: the rows before it,
    whose tokens share a tile with it, do not see them; it and the rows after
    it do."""
    for what in (float("nan"),) if ct == F8 else (float("nan"), float("inf"), -float("inf")):
        p = KvProblem([4], [70], H=2, G=2, D=64, page=16, q_dtype=qt, dtype=ct)
        clean = p.reference()
        page, slot = int(p.table[0, 68 // 16]), 68 % 16
        vf = p.v.float()
        vf[page, slot] = what
        p.v = vf.to(ct)
        d = KvDevice(p)
        out, lse = d.attend()
        o = out.double().cpu().numpy()
        ref = {k: (x if np.isscalar(x) else x.copy()) for k, x in clean.items()}
        for x in ref.values():
            if isinstance(x, np.ndarray) and x.ndim == 3:
                x[2:] = 0
        got = out.clone()
        got[2:] = 0
        p.check(got, None, ref, f"rows before a {what}")
        assert np.isfinite(o[:2]).all()
        if what != what:
            assert np.isnan(o[2:]).all()
        else:
            assert (o[2:] == what).all()
        # the same in a key: its row's scores are NaN or infinite from there on
        p = KvProblem([4], [70], H=2, G=2, D=64, page=16, q_dtype=qt, dtype=ct)
        kf = p.k.float()
        kf[page, slot] = what
        p.k = kf.to(ct)
        out, lse = KvDevice(p).attend()
        got = out.clone()
        got[2:] = 0
        p.check(got, None, ref, f"rows before a key of {what}")
        assert torch.isnan(out[2:].float()).all()


@pytest.mark.parametrize("ct,D,M,G", [(BF, 64, 16, 9), (BF, 128, 9, 12), (F8, 128, 16, 6), (BF, 256, 8, 6), (F8, 256, 16, 5)])
def test_what_unseen_slots_hold_does_not_matter_where_waves_split_the_rows(ct, D, M, G):
    """More rows than one wave takes: the second last row's own value is NaN."""
    p = KvProblem([M], [300], H=2, G=G, D=D, page=16, dtype=ct, seed=D + G)
    clean = p.reference()
    j = 300 - 2
    vf = p.v.float()
    vf[int(p.table[0, j // 16]), j % 16] = float("nan")
    p.v = vf.to(ct)
    out, lse = KvDevice(p).attend()
    got, ref = out.clone(), dict(clean, out=clean["out"].copy(), mass=clean["mass"].copy())
    got[M - 2:], ref["out"][M - 2:], ref["mass"][M - 2:] = 0, 0, 0
    p.check(got, None, ref, "rows before a NaN")
    assert torch.isnan(out[M - 2:].float()).all()
    p.check(torch.zeros_like(out), lse, dict(clean, out=np.zeros_like(clean["out"])), "lse")


def test_large_scores():
    # scores of some thousands: weights of 0 and 1, no overflow
    p = KvProblem([3], [200], H=2, G=2, D=128, page=16, spread=400.0)
    parity(p, "large scores")
    p = KvProblem([3], [200], H=2, G=2, D=128, page=16)
    p.k = (p.k.float() - 40.0 * p.q[0, 0].float().sign()).to(BF)  # the first query's scores lie far below 0
    parity(p, "scores far below zero")


def test_strided_queries_outputs_and_caches():
    p = KvProblem([3, 2], [100, 37], H=2, G=3, D=128, page=16)
    ref = p.reference()
    qkv = torch.randn(p.T, 10, 128).to(BF)
    qkv[:, :6] = p.q
    x = qkv.cuda()
    d = KvDevice(p)
    d.q = x[:, :6]
    wide = torch.full((p.T, 9, 128), 7.0, dtype=BF, device="cuda")
    out, lse = d.attend(out=wide[:, 2:8])
    p.check(out, lse, ref, "slices")
    assert (wide[:, :2] == 7).all() and (wide[:, 8:] == 7).all()
    k, v = (t.cuda().transpose(1, 2).contiguous().transpose(1, 2) for t in (p.k, p.v))
    d.cache = q.KvCache(k, v, d.table)
    p.check(*d.attend(), ref, "head-major pages")
    kv = torch.stack([p.k, p.v], 1).cuda()
    d.cache = q.KvCache(kv[:, 0], kv[:, 1], d.table)
    p.check(*d.attend(), ref, "keys and values in one allocation")
    heads_first = torch.empty(6, p.T, 128, dtype=BF, device="cuda").transpose(0, 1)
    out, _ = d.attend(out=heads_first)
    p.check(out, None, ref, "output with heads first")


def test_offsets_past_32_bits():
    page, H, D = 64, 8, 128
    P = (5 << 30) // (page * H * D * 2)
    p = KvProblem([2, 3], [150, 97], H=H, G=2, D=D, page=page)
    k, v = (torch.empty(P, page, H, D, dtype=BF, device="cuda") for _ in range(2))
    move = torch.full((p.P,), -1, dtype=torch.long)
    used = p.table[p.table >= 0].long()
    move[used] = P - 1 - torch.arange(len(used)) * 2
    for i in used.tolist():
        k[move[i]], v[move[i]] = p.k[i].cuda(), p.v[i].cuda()
    d = KvDevice(p)
    table = torch.where(p.table >= 0, move[p.table.clamp(min=0).long()].to(torch.int32), p.table).cuda()
    d.cache = q.KvCache(k, v, table)
    p.check(*d.attend(), label="5 GiB caches")
    new = torch.randn(p.T, H, D)
    q.append(d.cache, new.cuda(), new.cuda(), d.start, d.len)
    torch.cuda.synchronize()
    last = int(table[1, 96 // page])
    assert last * page * H * D > 2 ** 31 and torch.equal(k[last, 96 % page].cpu(), new[4].to(BF))


def test_attend_repeats_bit_for_bit_and_without_workspace():
    p = KvProblem([5, 4, 5], [4000, 33, 900], H=4, G=6, D=128, page=16)
    d = KvDevice(p)
    work = q.attend_workspace(d.cache, p.M, p.H * p.G, p.T)
    a, za = d.attend(workspace=work)
    work.fill_(255)  # its contents are free
    b, zb = d.attend(workspace=work)
    c, _ = d.attend(lse=None)
    assert torch.equal(a, b) and torch.equal(za, zb) and torch.equal(a, c)
    with pytest.raises(q.QgemvError):
        d.attend(workspace=work[:8])


def test_attend_on_another_stream():
    p = KvProblem([5, 4], [3000, 500], H=4, G=6, D=128, page=16)
    d = KvDevice(p)
    want, _ = d.attend()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = q.attend(d.cache, d.q, d.start, d.len, p.M, scale=p.scale, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_step_in_a_graph():
    """append, attend and verify captured once and replayed on new rows, with
    eager work between the replays."""
    p = KvProblem([4, 3], [700, 90], H=2, G=4, D=128, page=16)
    d, eager = KvDevice(p), KvDevice(p)
    new_k, new_v = torch.zeros(p.T, 2, 128, device="cuda"), torch.zeros(p.T, 2, 128, device="cuda")
    pr, dr, tok, u, _ = draft_problem(p.rows, 3001)
    pr, dr, tok, u = pr.cuda(), dr.cuda(), tok.cuda(), u.cuda()
    work = q.attend_workspace(d.cache, p.M, 8, p.T)
    vwork = q.verify_workspace(pr, p.B)

    def step(x, w, vw):
        q.append(x.cache, new_k, new_v, x.start, x.len)
        o = q.attend(x.cache, x.q, x.start, x.len, p.M, scale=p.scale, workspace=w)
        return (o, *q.verify(pr, dr, tok, u, x.start, p.M, workspace=vw))

    step(d, work, vwork)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(d, work, vwork)
    for i in range(4):
        new_k.normal_()
        new_v.normal_()
        u.uniform_()
        d.q.normal_()
        eager.q.copy_(d.q)
        want = step(eager, None, None)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), f"replay {i}"
        assert same_bits(d.k, eager.k) and same_bits(d.v, eager.v)


# ---------------------------------------------------------------- verify

def check_verify(p, d, tokens, u, start, M=None, label=""):
    say(f"verify {label}")
    rows = (start[1:] - start[:-1]).tolist()
    f = lambda x: None if x is None else x.double().numpy()  # noqa: E731
    want, count, edges = oracle.verify_reference(f(p), f(d), tokens.tolist(), u.tolist(), start.tolist())
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    out, n = q.verify(c(p), c(d), c(tokens), c(u), c(start), M or max(max(rows), 1))
    torch.cuda.synchronize()
    out, n = out.cpu().numpy(), n.cpu().numpy()
    assert np.array_equal(n, count), label
    for b, e in enumerate(edges):
        if e is None:
            continue
        a, z = int(start[b]), int(start[b + 1])
        i = a + count[b] - 1
        before, upto, share, total = e
        # fp64 sums in another order: off by at most a step of 2^-52 per term
        slack = p.shape[1] * 2.0 ** -52 * total
        if share - before > slack and upto - share > slack:
            assert np.array_equal(out[a:z], want[a:z]), f"{label}: sequence {b}"
        else:
            assert np.array_equal(out[a:i], want[a:i]) and (out[i + 1:z] == -1).all()
            assert 0 <= out[i] < p.shape[1]
    return out, n


@pytest.mark.parametrize("dtype", [torch.float32, BF, HF])
@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("V", [1, 2, 63, 64, 255, 1000, 4097, 32000, 50257])
def test_verify(dtype, drafts, V):
    for seed in range(3):
        x = draft_problem([4, 1, 5, 16, 2, 3, 8], V, dtype, drafts, seed=seed + V)
        check_verify(*x, label=f"{dtype} drafts={drafts} V={V} seed={seed}")


def test_verify_one_sequence_and_large_vocabulary():
    check_verify(*draft_problem([5], 151936, seed=2), label="V=151936")
    check_verify(*draft_problem([1], 131073, BF, False, seed=2), label="one row")


def test_verify_many_sequences():
    check_verify(*draft_problem([1 + b % 4 for b in range(300)], 777, seed=1), label="300 sequences")
    check_verify(*draft_problem([b % 3 for b in range(40)], 500, seed=1), label="sequences without rows")


def test_verify_edges_of_the_draw():
    """Numbers of 0 and just below 1, probabilities with long runs of zeros,
    all weight on one token, nothing left after a refusal."""
    V = 3001
    for u1 in (0.0, 0.5, 1.0 - 2.0 ** -24):
        for hot in ((0,), (V - 1,), (1500,), (700, 2300)):
            p = torch.zeros(2, V)
            p[:, list(hot)] = 1.0 / len(hot)
            tok = torch.tensor([0, 5], dtype=torch.int32)
            u = torch.tensor([0.5, u1])
            start = torch.tensor([0, 2], dtype=torch.int32)
            out, n = check_verify(p, None, tok, u, start, label=f"u={u1} hot={hot}")
            assert n[0] == 1 and out[0] == (hot[0] if u1 < 0.5 or len(hot) == 1 else hot[1])
    # the draft holds all of p's weight: refused only where u * q is not below p
    p = torch.zeros(2, V)
    p[:, 9] = 1.0
    d = p.clone()
    out, n = check_verify(p, d, torch.tensor([0, 9], dtype=torch.int32), torch.tensor([0.999, 0.3]),
                          torch.tensor([0, 2], dtype=torch.int32), label="p = q")
    assert n[0] == 2 and out.tolist() == [9, 9]
    d[:, 9], d[:, 10] = 1.0, 0.0
    d[0, 10] = 1.0  # refused (p is 0 there) and nothing left of p - q
    out, n = check_verify(p, d, torch.tensor([0, 10], dtype=torch.int32), torch.tensor([0.2, 0.3]),
                          torch.tensor([0, 2], dtype=torch.int32), label="nothing left")
    assert n[0] == 1 and out.tolist() == [9, -1]


def test_verify_accepts_by_exact_products():
    """u * q against p one step of fp32 apart: the product is not rounded."""
    u = torch.tensor([1.0 - 2.0 ** -24, 0.5])
    qv = torch.tensor(1.0 / 3.0)
    prod = float(u[0].double() * qv.double())
    start = torch.tensor([0, 2], dtype=torch.int32)
    near = torch.tensor(prod, dtype=torch.float64).float()
    for pv in (near, torch.nextafter(near, torch.tensor(0.0)), torch.nextafter(near, torch.tensor(1.0))):
        p, d = torch.full((2, 4), 0.1), torch.full((2, 4), 0.2)
        p[0, 2], d[0, 2] = pv, qv
        _, n = check_verify(p, d, torch.tensor([0, 2], dtype=torch.int32), u, start, label="product")
        assert n[0] == (2 if prod < float(pv) else 1)


def test_verify_odd_inputs():
    V = 500
    p, d, tok, u, start = draft_problem([3, 3, 3], V, seed=4)
    tok[1], tok[4], tok[7] = -1, V, 2 ** 31 - 1  # drafts outside the vocabulary are refused
    _, n = check_verify(p, d, tok, u, start, label="drafts out of range")
    assert n.tolist() == [1, 1, 1]
    check_verify(p, None, tok, u, start, label="drafts out of range, no probabilities")
    # sums that are NaN give token 0, sums of nothing the last
    x = torch.full((1, V), float("nan"))
    s = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _ = q.verify(x.cuda(), None, one, torch.tensor([0.5], device="cuda"), s, 1)
    assert out.tolist() == [0]
    out, _ = q.verify(torch.zeros_like(x).cuda(), None, one, torch.tensor([0.5], device="cuda"), s, 1)
    assert out.tolist() == [V - 1]


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_verify_strided_rows(dtype):
    """Rows that start at any element: another stride for p than for q."""
    p, d, tok, u, start = draft_problem([4, 2, 5], 1001, dtype, seed=3)
    want = q.verify(p.cuda(), d.cuda(), tok.cuda(), u.cuda(), start.cuda(), 5)
    a = torch.zeros(11, 1024, dtype=dtype, device="cuda")
    b = torch.zeros(11, 1003, dtype=dtype, device="cuda")
    a[:, 3:1004], b[:, 1:1002] = p.cuda(), d.cuda()
    got = q.verify(a[:, 3:1004], b[:, 1:1002], tok.cuda(), u.cuda(), start.cuda(), 5)
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_verify_repeats_on_one_workspace():
    p, d, tok, u, start = (x.cuda() for x in draft_problem([4, 2, 5, 1], 9001, seed=3))
    work = q.verify_workspace(p, 4)
    want = q.verify(p, d, tok, u, start, 5, workspace=work)
    for _ in range(5):
        got = q.verify(p, d, tok, u, start, 5, workspace=work)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = q.verify(p, d, tok, u, start, 5, workspace=work, stream=s)
    s.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_verify_calls_of_several_sizes_share_a_workspace():
    sizes = [([5], 40000), ([2] * 300, 1500), ([4, 3, 1] * 9, 9001), ([3] * 1500, 70), ([16, 1], 300001)]
    problems = [draft_problem(rows, V, seed=V) for rows, V in sizes]
    need = max(q.lib().qgemv_verify_drafts_workspace(len(rows), V) for rows, V in sizes)
    work = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for i in range(3):
        for (rows, V), x in zip(sizes, problems):
            args = [t.cuda() for t in x]
            want = q.verify(*args, max(rows))
            got = q.verify(*args, max(rows), workspace=work)
            assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]), (i, len(rows), V)


def test_verify_does_not_depend_on_the_other_sequences():
    """A sequence's answer is the same alone and among others, where other
    numbers of workgroups share it."""
    p, d, tok, u, start = (x.cuda() for x in draft_problem([4, 2, 7, 1] * 30, 20011, seed=8))
    out, n = q.verify(p, d, tok, u, start, 7)
    for b in (0, 1, 2, 3, 61, 119):
        s, e = int(start[b]), int(start[b + 1])
        one = torch.tensor([0, e - s], dtype=torch.int32, device="cuda")
        o, m = q.verify(p[s:e], d[s:e], tok[s:e].clone(), u[s:e].clone(), one, 7)
        assert torch.equal(o, out[s:e]) and torch.equal(m, n[b:b + 1])
