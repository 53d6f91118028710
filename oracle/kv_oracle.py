"""fp64 CPU oracle of the verify step's cache append, attention and draft
acceptance.

TEST INFRASTRUCTURE ONLY, as :mod:`oracle.qgemv_oracle`: it shares no code
with the HIP path and imports nothing from the product package.  Inputs are
float64 or integer numpy arrays (16- and 8-bit values are exact in fp64); the
definitions are written out sequence by sequence and row by row.
"""
from __future__ import annotations

import numpy as np

__all__ = ["row_places", "slot_of", "append_places", "visible", "attend_reference", "verify_weights",
           "verify_reference", "round_e4m3"]


def row_places(start, length):
    """(row, sequence, position) of every row that has a sequence."""
    out = []
    for b, n in enumerate(length):
        for t in range(int(start[b]), int(start[b + 1])):
            out.append((t, b, int(n) - (int(start[b + 1]) - t)))
    return out


def slot_of(table, b: int, j: int, page: int, pages: int):
    """(page id, slot) of token j of sequence b, or None where there is none."""
    if j < 0 or j // page >= table.shape[1]:
        return None
    i = int(table[b, j // page])
    return (i, j % page) if 0 <= i < pages else None


def append_places(table, start, length, page: int, pages: int):
    """(row, page id, slot) of every row that append writes."""
    out = []
    for t, b, pos in row_places(start, length):
        s = slot_of(table, b, pos, page, pages)
        if s is not None:
            out.append((t, *s))
    return out


def round_e4m3(x) -> np.ndarray:
    """Values limited to +-448 and rounded to the nearest E4M3 number, ties to
    the even significand; NaN stays."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where(a > 0, np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    step = np.exp2(np.maximum(e, -6.0) - 3.0)  # 3 bits after the leading one; subnormals share 2^-9
    r = np.rint(a / step) * step  # rint: ties to even
    return np.where(np.isnan(x), np.nan, np.copysign(r, x))


def visible(pos: int, length: int, window: int, sinks: int) -> np.ndarray:
    """The tokens that the row at `pos` sees, ascending."""
    j = np.arange(max(0, min(pos + 1, length)))
    if window:
        j = j[(j > pos - window) | (j < sinks)]
    return j


def attend_reference(q, k, v, table, start, length, window=0, sinks=0, scale=1.0, k_scale=None, v_scale=None):
    """q [T, Hq, D], k and v [pages, page, H, D].  Returns a dict of
      out [T, Hq, D], lse [T, Hq];
      mass [T, Hq, D]: sum of p_j |v_j| (p the normalized weights);
      size [T, Hq]: the largest scale * sum_d |q_d k_jd| of a seen token;
      count [T]: how many tokens the row sees;
      top [H, D] largest |v| of a seen token's column.
    Rows that see nothing: 0, -inf."""
    T, Hq, D = q.shape
    P, page, H, _ = k.shape
    G = Hq // H
    out, mass = np.zeros(q.shape), np.zeros(q.shape)
    lse, size = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    count = np.zeros(T, np.int64)
    vmax = 0.0
    for t, b, pos in row_places(start, length):
        where = [s for s in (slot_of(table, b, int(j), page, P) for j in visible(pos, int(length[b]), window, sinks))
                 if s is not None]
        count[t] = len(where)
        if not where:
            continue
        ids, slots = np.array(where).T
        for h in range(H):
            kk = k[ids, slots, h] * (1.0 if k_scale is None else float(k_scale[h]))
            vv = v[ids, slots, h] * (1.0 if v_scale is None else float(v_scale[h]))
            with np.errstate(invalid="ignore"):
                vmax = max(vmax, float(np.nanmax(np.abs(vv))))
                for hq in range(h * G, (h + 1) * G):
                    s = (kk @ q[t, hq]) * scale
                    top = s.max()
                    e = np.exp(s - top)
                    total = e.sum()
                    lse[t, hq] = top + np.log(total)
                    out[t, hq] = (e @ vv) / total
                    mass[t, hq] = (e @ np.abs(vv)) / total
                    size[t, hq] = (np.abs(kk) @ np.abs(q[t, hq])).max() * abs(scale)
    return {"out": out, "lse": lse, "mass": mass, "size": size, "count": count, "top": vmax}


def verify_weights(p, q, tokens, u, a: int, e: int):
    """Rows a..e-1 of one sequence: (accepted drafts, weights the next token is
    drawn from)."""
    t = a
    V = p.shape[1]
    while t < e - 1:
        d = int(tokens[t + 1])
        if not 0 <= d < V:
            break
        if not float(u[t]) * (1.0 if q is None else float(q[t, d])) < float(p[t, d]):
            break
        t += 1
    w = p[t].copy()
    if t < e - 1:
        if q is not None:
            w = np.maximum(w - q[t], 0.0)
        elif 0 <= int(tokens[t + 1]) < V:
            w[int(tokens[t + 1])] = 0.0
        if not w.sum() > 0:
            w = p[t].copy()
    return t - a, w


def verify_reference(p, q, tokens, u, start):
    """Returns (out [T], count [B], edges): edges[b] = (running sums up to and
    with the drawn token, the number it was compared with, sum)."""
    out = np.full(p.shape[0], -1, np.int64)
    count, edges = [], []
    for a, e in zip(start[:-1], start[1:]):
        a, e = int(a), int(e)
        if e <= a:
            count.append(0)
            edges.append(None)
            continue
        n, w = verify_weights(p, q, tokens, u, a, e)
        c = np.cumsum(w)
        share = float(u[e - 1]) * c[-1]
        i = min(int(np.searchsorted(c, share, side="right")), len(c) - 1)
        out[a:a + n] = tokens[a + 1:a + 1 + n]
        out[a + n] = i
        count.append(n + 1)
        edges.append((c[i - 1] if i else 0.0, c[i], share, c[-1]))
    return out, np.array(count), edges
