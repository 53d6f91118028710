"""Pins for the oracle's cache append, attention and draft acceptance, against
closed forms and exact arithmetic, with planted mistakes that must fail."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle import kv_oracle

from kv_util import KvProblem, draft_problem


def test_places_follow_the_table():
    table = np.array([[4, 1, -1], [2, 0, 9]])
    # sequence 0: 2 rows, 5 tokens, pages of 3; sequence 1: 3 rows, 2 tokens (a row before the first)
    got = oracle.append_places(table, [0, 2, 5], [5, 2], 3, 5)
    assert got == [(0, 1, 0), (1, 1, 1), (3, 2, 0), (4, 2, 1)]
    assert kv_oracle.slot_of(table, 0, 7, 3, 5) is None   # a page that is not there
    assert kv_oracle.slot_of(table, 1, 6, 3, 5) is None   # an id past the pages
    assert kv_oracle.slot_of(table, 1, 9, 3, 5) is None   # past the table


@pytest.mark.parametrize("window,sinks,want", [
    (0, 0, [0, 1, 2, 3, 4, 5]), (0, 3, [0, 1, 2, 3, 4, 5]), (2, 0, [4, 5]), (2, 1, [0, 4, 5]),
    (2, 9, [0, 1, 2, 3, 4, 5]), (1, 0, [5]), (100, 0, [0, 1, 2, 3, 4, 5]),
])
def test_visible_tokens(window, sinks, want):
    assert oracle.visible(5, 8, window, sinks).tolist() == want
    assert oracle.visible(-1, 8, window, sinks).tolist() == []
    assert oracle.visible(5, 0, window, sinks).tolist() == []


def test_e4m3_rounding_is_the_types():
    g = torch.Generator().manual_seed(3)
    x = torch.cat([torch.randn(4000, generator=g) * s for s in (1e-3, 1.0, 60.0, 400.0)])
    x = torch.cat([x, torch.arange(0, 256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()])
    x = x[~x.isnan()].clamp(-448, 448)
    assert np.array_equal(oracle.round_e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())
    assert oracle.round_e4m3([1e9, -np.inf]).tolist() == [448.0, -448.0] and np.isnan(oracle.round_e4m3(np.nan))
    # ties to even: 17 lies between 16 and 18, 19 between 18 and 20
    assert oracle.round_e4m3([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10]).tolist() == [16.0, 20.0, 0.0, 2.0 ** -8]


def test_equal_scores_give_the_mean_and_the_count():
    p = KvProblem([2, 3], [9, 21], H=2, G=3, D=64, page=5, window=6, sinks=2)
    p.q.zero_()
    r = p.reference()
    for t, b, pos in kv_oracle.row_places(p.start.tolist(), p.lens):
        js = oracle.visible(pos, p.lens[b], 6, 2)
        assert r["count"][t] == len(js)
        for h in range(2):
            vv = np.mean([p.v[p.table[b, j // 5], j % 5, h].double().numpy() for j in js], axis=0)
            assert np.allclose(r["out"][t, h * 3:(h + 1) * 3], vv, rtol=0, atol=1e-14)
        assert np.allclose(r["lse"][t], np.log(len(js)), rtol=0, atol=1e-13)


def test_one_large_score_selects_its_value():
    p = KvProblem([1], [40], H=1, G=1, D=64, page=7)
    j = 17
    p.q[0, 0] = (20.0 * p.k[p.table[0, j // 7], j % 7, 0].float()).to(p.q.dtype)
    r = p.reference()
    assert np.allclose(r["out"][0, 0], p.v[p.table[0, j // 7], j % 7, 0].double().numpy(), atol=1e-12)


def test_attend_matches_a_direct_sum_and_planted_mistakes_do_not():
    p = KvProblem([3, 2], [11, 30], H=2, G=2, D=64, page=4, dtype=torch.float8_e4m3fn, window=9, sinks=1, seed=5)
    r = p.reference()

    def direct(shift=0, swap=False, drop_scale=False):
        out = np.zeros_like(r["out"])
        for t, b, pos in kv_oracle.row_places(p.start.tolist(), p.lens):
            for hq in range(4):
                h = hq % 2 if swap else hq // 2
                num, den = np.zeros(64), 0.0
                for j in range(pos + 1 + shift):
                    if not (j > pos - 9 or j < 1) or j >= p.lens[b]:
                        continue
                    s = int(p.table[b, j // 4]), j % 4, h
                    w = np.exp(p.scale * float(p.k_scale[h]) * float(p.q[t, hq].double() @ p.k[s].double()))
                    num += w * p.v[s].double().numpy() * (1.0 if drop_scale else float(p.v_scale[h]))
                    den += w
                out[t, hq] = num / den
        return out

    assert np.allclose(direct(), r["out"], rtol=1e-12, atol=1e-13)
    for bad in (dict(shift=1), dict(swap=True), dict(drop_scale=True)):
        assert not np.allclose(direct(**bad), r["out"], rtol=1e-3, atol=1e-3)
    assert (r["mass"] + 1e-12 >= np.abs(r["out"])).all()


def test_verify_closed_forms():
    p = np.array([[0.5, 0.25, 0.25], [0.1, 0.6, 0.3], [0.2, 0.2, 0.6]])
    q = np.array([[0.25, 0.5, 0.25], [0.1, 0.6, 0.3], [1.0, 0.0, 0.0]])
    # row 0's draft is token 1: accepted iff u < 0.5
    out, count, _ = oracle.verify_reference(p, q, [0, 1, 1], [0.49, 0.9, 0.0], [0, 3])
    assert out.tolist() == [1, 1, 0] and count.tolist() == [3]  # p == q accepts; the draw from p[2] at 0
    out, count, _ = oracle.verify_reference(p, q, [0, 1, 1], [0.5, 0.9, 0.99], [0, 3])
    assert out.tolist() == [0, -1, -1] and count.tolist() == [1]  # what is left of row 0 is token 0
    out, _, _ = oracle.verify_reference(p, None, [0, 2, 1], [0.3, 0.9, 0.5], [0, 3])
    assert out.tolist() == [0, -1, -1]  # token 2 refused: 0.5 and 0.25 are left, half way is token 0
    out, _, _ = oracle.verify_reference(p, None, [0, 2, 1], [0.3, 0.9, 0.7], [0, 3])
    assert out.tolist() == [1, -1, -1]
    same = np.array([[0.5, 0.5], [1.0, 0.0]])
    out, _, _ = oracle.verify_reference(same, same, [0, 5], [0.0, 0.75], [0, 2])
    assert out.tolist() == [1, -1]  # a draft outside the vocabulary; nothing left: drawn from p
    assert oracle.verify_reference(p, None, [0, 2, 1], [0.3, 0.9, 0.7], [0, 0, 3])[1].tolist() == [0, 1]


def test_verify_draw_matches_exact_sums():
    p, q, tokens, u, start = draft_problem([4, 1, 3], 50, seed=8)
    out, count, _ = oracle.verify_reference(p.double().numpy(), q.double().numpy(), tokens.tolist(), u.tolist(),
                                            start.tolist())
    for b in range(3):
        a, e = int(start[b]), int(start[b + 1])
        n = int(count[b]) - 1
        w = [Fraction(float(x)) for x in p[a + n]]
        if a + n < e - 1:
            w = [max(x - Fraction(float(y)), Fraction(0)) for x, y in zip(w, q[a + n])]
        share, run = Fraction(float(u[e - 1])) * sum(w), Fraction(0)
        for i, x in enumerate(w):
            run += x
            if run > share:
                break
        assert out[a + n] == i
