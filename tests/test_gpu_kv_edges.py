"""GPU tests of the cache append, the attention and the draft acceptance at
borders: the table's end, starts out of order, sums that round, weights far
below the largest, a stream given by its address."""
import numpy as np
import pytest
import torch

import oracle
from few_row_quantized_amd import qgemv as q

from gpu_util import say
from kv_util import STEP, KvDevice, KvProblem, draft_problem

pytestmark = pytest.mark.gpu
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu(require_gpu):
    torch.cuda.init()
    yield


# ---------------------------------------------------------------- lengths past the table

def past_the_table(rows, lens, over, **kw):
    """A problem whose sequences b have over[b] tokens more than the pages that
    were laid out for them; the table is as wide as the longest."""
    p = KvProblem(rows, lens, extra_width=0, **kw)
    p.lens = [n + x for n, x in zip(lens, over)]
    p.len = torch.tensor(p.lens, dtype=torch.int32)
    p.poison()
    return p


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (5, 2), (40, 0), (64, 33), (5000, 4)])
@pytest.mark.parametrize("qt,ct,D,G", [(BF, BF, 128, 2), (HF, F8, 64, 3), (BF, BF, 128, 20)])
def test_rows_past_the_tables_end(qt, ct, D, G, window, sinks):
    """Rows stand at len - rows and on, whether or not the table reaches there:
    the first of them may fit (and see themselves), the others see what is
    there.  One sequence ends before the table's end, with pages missing."""
    say(f"attend past the table {qt} {ct} D={D} G={G} window={window} sinks={sinks}")
    p = past_the_table([5, 5, 2, 4, 3], [96, 96, 96, 96, 40], [4, 1, 2, 90, 20], H=2, G=G, D=D, page=16, q_dtype=qt,
                       dtype=ct, window=window, sinks=sinks, seed=window + G)
    p.check(*KvDevice(p).attend(), label="past the table")


@pytest.mark.parametrize("window,sinks", [(0, 0), (1000, 5)])
@pytest.mark.parametrize("G", [4, 20])
def test_rows_past_the_end_of_a_long_table(G, window, sinks):
    say(f"attend past a long table G={G} window={window}")
    p = past_the_table([5, 3, 4], [4800, 4800, 700], [3, 700, 0], H=2, G=G, D=64, page=16, window=window, sinks=sinks,
                       seed=G)
    p.check(*KvDevice(p).attend(), label="past a long table")


@pytest.mark.parametrize("G", [2, 20])
def test_lengths_far_past_the_table(G):
    """Up to the largest int32: all of the table without a window, with one the
    sinks, or nothing."""
    for window, sinks in ((0, 0), (7, 0), (7, 40), (2 ** 30, 0), (2 ** 31 - 1, 3)):
        say(f"attend far past the table G={G} window={window}")
        p = past_the_table([2, 3], [64, 50], [500, 500], H=1, G=G, D=64, page=16, window=min(window, 2 ** 29), sinks=sinks)
        p.window = window
        d = KvDevice(p)
        ref = p.reference()
        far = (10 ** 9, 2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1) if window < 100 else ()
        for n in (0, *far):
            if n:
                d.len = torch.tensor([n, n], dtype=torch.int32, device="cuda")
            p.check(*d.attend(), ref, label=f"length {n}")
        if window == 7 and sinks == 0:
            assert np.isneginf(ref["lse"]).all()


def test_a_row_appended_to_the_last_slot_sees_itself():
    """96 slots, a length of 100, 5 rows: the first is appended to slot 95 and
    attends up to there; the four after it are dropped and see the same."""
    p = past_the_table([5], [96], [4], H=2, G=2, D=64, page=16, spare=0)
    d = KvDevice(p)
    g = torch.Generator().manual_seed(3)
    new_k, new_v = (torch.randn((5, 2, 64), generator=g) for _ in range(2))
    q.append(d.cache, new_k.cuda(), new_v.cuda(), d.start, d.len)
    page, slot = int(p.table[0, 5]), 15
    p.k[page, slot], p.v[page, slot] = new_k[0].to(BF), new_v[0].to(BF)
    assert torch.equal(d.k.cpu(), p.k) and torch.equal(d.v.cpu(), p.v)
    p.check(*d.attend(), label="after the append")


# ---------------------------------------------------------------- draws at rounding borders

def weights_at_a_border(V, at):
    p = torch.zeros(1, V)
    for i, w in at.items():
        p[0, i] = w
    return p


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("V,u,at", [
    # 1/2 and twice 2^-54, which round to nothing one by one and to a step of
    # the sum together: where a sum over no weight at all first sees both
    (600, 0.5, {14: 0.5, 16: 2.0 ** -54, 20: 2.0 ** -54, 550: 0.5}),
    # the same over the 512-token pieces of a row
    (30000, 0.5, {7 * 512: 0.5, 8 * 512: 2.0 ** -54, 10 * 512: 2.0 ** -54, 40 * 512: 0.5}),
    # four tokens a thread: the sum before them, taken back from the sum after
    # them, is a step above the number that is looked for
    (140000, 2.0 ** -61, {40: 0.5, 61: 0.5, 62: 2.0 ** -52, 63: 2.0 ** -53, 139000: 2.0 ** 60}),
])
def test_no_token_without_weight_is_drawn(dtype, V, u, at):
    p = weights_at_a_border(V, at).to(dtype)
    for lead in (0, 1, 2, 3, 5):  # also at other places of a thread and a load
        x = torch.roll(p, lead, 1)
        say(f"verify border V={V} {dtype} lead={lead}")
        one = torch.zeros(1, dtype=torch.int32, device="cuda")
        start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        out, n = q.verify(x.cuda(), None, one, torch.tensor([u], device="cuda"), start, 1)
        assert n.tolist() == [1]
        i = int(out[0])
        assert float(x[0, i]) > 0.0, f"token {i} has no weight (at lead {lead})"
        # and the sum up to it is the number that is looked for, to a few steps
        c = torch.cumsum(x[0].double(), 0)
        share, slack = u * float(c[-1]), 16 * 2.0 ** -52 * max(u * float(c[-1]), 0.5)
        assert float(c[i]) >= share - slack and float(c[i] - x[0, i].double()) <= share + slack


# ---------------------------------------------------------------- one workspace for smaller calls

def test_fewer_rows_on_the_workspace_of_more():
    """Sized once for the most rows of a step, as a serving loop does: 10 rows
    need no parts over this table, fewer do."""
    B = 32
    lens = [2000] + [400 - 11 * b for b in range(1, B)]
    work = None
    for M in (10, 8, 1, 5, 2):
        say(f"attend M={M} on the workspace of 10")
        p = KvProblem([M] * B, lens, H=4, G=6, D=128, page=16, seed=M, extra_width=0)
        d = KvDevice(p)
        if work is None:
            work = q.attend_workspace(d.cache, 10, 24, 10 * B)
        p.check(*d.attend(workspace=work), label=f"M={M}")


# ---------------------------------------------------------------- streams by address

def test_stream_zero_is_the_default_stream():
    """0 is the default stream's address; torch's ExternalStream(0) would be a
    stream of its pool, which waits for nothing."""
    from few_row_quantized_amd import kv
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        with kv._allocating(0, torch.device("cuda", 0)):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
        with kv._allocating(side.cuda_stream, torch.device("cuda", 0)):
            assert torch.cuda.current_stream().cuda_stream == side.cuda_stream
    x = [t.cuda() for t in draft_problem([4, 2, 5], 9001, seed=3)]
    p = KvProblem([5, 4], [3000, 500], H=4, G=6, D=128, page=16)
    d = KvDevice(p)
    want, want_out = q.verify(*x, 5), d.attend()[0]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = q.verify(*x, 5, stream=0)
        out = q.attend(d.cache, d.q, d.start, d.len, p.M, scale=p.scale, stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(out, want_out)


# ---------------------------------------------------------------- starts out of order or out of range

def test_starts_are_limited_alike_by_append_and_attention():
    """start below 0 or past the rows counts as 0 or T: the rows in between are
    placed as by starts within them, in the cache and in the attention."""
    for start, same in (([-5, 2, 900], [0, 2, 4]), ([-1, -1, 2 ** 31 - 1], [0, 0, 4]), ([1, 9, 9], [1, 4, 4]),
                        ([-2 ** 31, 3, 2 ** 31 - 1], [0, 3, 4])):
        say(f"starts {start}")
        p = KvProblem([2, 2], [40, 50], H=1, G=2, D=64, page=16)
        g = torch.Generator().manual_seed(1)
        new_k, new_v = (torch.randn((4, 1, 64), generator=g) for _ in range(2))
        p.start = torch.tensor(same, dtype=torch.int32)
        for t, i, s in oracle.append_places(p.table.numpy(), same, p.lens, p.page, p.P):
            p.k[i, s], p.v[i, s] = new_k[t].to(BF), new_v[t].to(BF)
        ref = p.reference()
        p = KvProblem([2, 2], [40, 50], H=1, G=2, D=64, page=16)
        d = KvDevice(p)
        d.start = torch.tensor(start, dtype=torch.int32, device="cuda")
        q.append(d.cache, new_k.cuda(), new_v.cuda(), d.start, d.len)
        want = KvProblem([2, 2], [40, 50], H=1, G=2, D=64, page=16)
        for t, i, s in oracle.append_places(want.table.numpy(), same, want.lens, want.page, want.P):
            want.k[i, s], want.v[i, s] = new_k[t].to(BF), new_v[t].to(BF)
        torch.cuda.synchronize()
        assert torch.equal(d.k.cpu(), want.k) and torch.equal(d.v.cpu(), want.v), start
        out = torch.zeros_like(d.q)
        lse = torch.full((4, 2), -float("inf"), device="cuda")
        d.attend(out=out, lse=lse, M=16)
        p.check(out, lse, ref, label=str(start))


def test_rows_of_descending_starts_write_nothing():
    """Sequence 1 ends before it begins: rows 3 and 4 are no longer its own, and
    no slot of it is written (nor any past its length)."""
    p = KvProblem([3, 2, 3], [20, 20, 20], H=1, G=1, D=64, page=16)
    new = torch.randn(8, 1, 64)
    want = p.k.clone()
    for t, b, pos in ((0, 0, 15), (1, 0, 16), (2, 0, 17), (5, 2, 17), (6, 2, 18), (7, 2, 19)):
        want[int(p.table[b, pos // 16]), pos % 16] = new[t].to(BF)
    d = KvDevice(p)
    d.start = torch.tensor([0, 5, 3, 8], dtype=torch.int32, device="cuda")
    q.append(d.cache, new.cuda(), new.cuda(), d.start, d.len)
    torch.cuda.synchronize()
    assert torch.equal(d.k.cpu(), want)


# ---------------------------------------------------------------- fp16: weights far below the largest

@pytest.mark.parametrize("ct", [HF, F8])
@pytest.mark.parametrize("M,G", [(1, 1), (2, 3), (16, 6)])
@pytest.mark.parametrize("B,n,nats", [(1, 131072, 18.0), (768, 65536, 18.0), (768, 20000, 17.0)])
def test_a_long_tail_below_one_large_weight(ct, M, G, B, n, nats):
    """The first token stands `nats` above a long, nearly uniform remainder and
    has a value of 0: the output is what the remainder contributes.  B sequences
    of the same pages, so that a workgroup walks long ranges.  The bound counts
    as KvProblem.check, but for weights below fp16's normal range: half of
    2^-24 absolute where the largest weight is at least 2^7, 2^-32 of it."""
    say(f"attend tail {ct} M={M} G={G} B={B} n={n}")
    p = KvProblem([M], [n], H=1, G=G, D=64, page=64, q_dtype=HF, dtype=ct, seed=n)
    g = torch.Generator().manual_seed(n)
    p.q.zero_()
    p.q[:, :, 0] = 16.0  # a score is 2 k[0]
    k, v = p.k.float(), p.v.float()
    k[..., 0] = 0.05 * torch.randn(k.shape[:3], generator=g)
    v.copy_(1.0 + 0.25 * torch.rand(v.shape, generator=g))
    first = int(p.table[0, 0]), 0
    k[first][:, 0], v[first] = nats / 2.0, 0.0
    if ct == F8:
        p.k_scale.fill_(1.0)
        p.v_scale.fill_(1.0)
    p.k, p.v = k.to(ct), v.to(ct)
    r = p.reference()
    d = KvDevice(p)
    d.cache = q.KvCache(d.k, d.v, d.table.repeat(B, 1).contiguous(), d.k_scale, d.v_scale)
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda") * M
    lse = torch.full((B * M, G), float("nan"), device="cuda")
    out = q.attend(d.cache, d.q.repeat(B, 1, 1), start, d.len.repeat(B), M, scale=p.scale, lse=lse)
    count = r["count"][:, None].astype(np.float64)
    weight = 2 * (p.D + 7) * 2.0 ** -24 * r["size"] + (2 * count + 16) * 2.0 ** -24
    u = STEP[HF]
    tol = u * np.abs(r["out"]) + (weight + u)[..., None] * (1 + u) * r["mass"] + 2.0 ** -25 \
        + 2.0 ** -32 * count[..., None] * r["top"]
    assert (np.abs(r["out"]) > 4 * tol).all()  # the tail is what is looked at
    off = np.abs(out.double().cpu().numpy().reshape(B, M, G, 64) - r["out"])
    assert (off <= tol).all(), f"off by {(off / tol).max()} of the bound, {off.max()} of {np.abs(r['out']).max()}"
    z = lse.double().cpu().numpy().reshape(B, M, G)
    assert (np.abs(z - r["lse"]) <= weight + 4 * 2.0 ** -24 * np.abs(r["lse"])).all()


@pytest.mark.parametrize("qt", [BF, HF])
def test_weights_stay_finite_where_scores_have_wide_steps(qt):
    """Scores past 2^27, whose fp32 steps are 16 and more: no weight passes the
    type's range, whatever order the largest come in."""
    for a, b in ((8, 16), (16, 8), (13, 27), (14, 28), (11, 50)):
        for step in (4.0, 8.0, 12.0, 16.0, 20.0, 24.0, 32.0):
            p = KvProblem([1], [129], H=1, G=1, D=64, page=16, q_dtype=qt)
            p.scale = 1.0
            p.q.zero_()
            p.q[0, 0, 0], p.q[0, 0, 1] = 2.0 ** 14, 1.0
            p.k.zero_()
            at = lambda j: (int(p.table[0, j // 16]), j % 16)  # noqa: E731
            for j in range(129):
                p.k[at(j)][0, 0] = a * 2.0 ** 9 + b
                p.k[at(j)][0, 1] = step * (j // 32)
            say(f"attend wide steps {qt} {a} {b} {step}")
            out, lse = KvDevice(p).attend()
            assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
            assert out.float().abs().max() <= p.v.float().abs().max() * (1 + 2 * STEP[qt])
