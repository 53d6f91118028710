"""fp64 CPU oracle of the rotation of positions, the routing to experts and the
adapters of a verify step.

TEST INFRASTRUCTURE ONLY, as :mod:`oracle.qgemv_oracle`: it shares no code
with the HIP path and imports nothing from the product package.  Inputs are
float64 or integer numpy arrays (16-bit values are exact in fp64); the
definitions are written out row by row.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["angle_reference", "rotate_reference", "route_reference", "adapt_reference"]


_BITS = 256  # after the point


def _pi() -> int:
    """pi in units of 2^-_BITS: 16 arctan(1/5) - 4 arctan(1/239)."""
    def arctan_of_one_over(n):
        term = total = (1 << (_BITS + 16)) // n
        i, sign = 3, -1
        while term:
            term //= n * n
            total += sign * (term // i)
            i, sign = i + 2, -sign
        return total
    return (16 * arctan_of_one_over(5) - 4 * arctan_of_one_over(239)) >> 16


_TURN = 2 * _pi()


def angle_reference(position, freq) -> float:
    """position * freq less whole turns, rounded once: the product and the turns
    in whole numbers, since neither fits fp64 where positions are far."""
    num, den = float(freq).as_integer_ratio()
    angle = (int(position) * num << _BITS) // den
    return math.ldexp(float(angle - (2 * angle + _TURN) // (2 * _TURN) * _TURN), -_BITS)


def rotate_reference(x, position, freq, axes=None, interleaved=False):
    """x [T, heads, dim] with the pairs of its values turned by position * freq:
    position [A][T] integers, freq [pairs], axes [pairs] or None (the first)."""
    y = np.array(x, dtype=np.float64)
    pairs = len(freq)
    for t in range(x.shape[0]):
        for i in range(pairs):
            axis = 0 if axes is None else min(max(int(axes[i]), 0), len(position) - 1)
            angle = angle_reference(position[axis][t], freq[i])
            c, s = math.cos(angle), math.sin(angle)
            p, q = (2 * i, 2 * i + 1) if interleaved else (i, pairs + i)
            a, b = np.array(x[t, :, p]), np.array(x[t, :, q])
            y[t, :, p], y[t, :, q] = a * c - b * s, a * s + b * c
    return y


def route_reference(logits, k, softmax=True, bias=None, groups=1, keep=1, best=1, renormalise=True, scale=1.0):
    """(experts [T, k], weights [T, k])."""
    T, E = logits.shape
    size = E // groups
    experts, weights = np.full((T, k), -1, np.int64), np.zeros((T, k))
    by_logit = bias is None and (best == 1 or groups == 1)
    for t in range(T):
        x = logits[t]
        there = [e for e in range(E) if x[e] > -math.inf]  # neither -inf nor NaN
        if not there:
            continue
        if softmax:
            top = max(x[e] for e in there)
            total = math.fsum(math.exp(x[e] - top) for e in there)
            score = {e: math.exp(x[e] - top) / total for e in there}
        else:
            score = {e: 1 / (1 + math.exp(-x[e])) if x[e] > -700 else math.exp(max(x[e], -745.2)) for e in there}
        choice = {e: x[e] if by_logit else score[e] + (0.0 if bias is None else bias[e]) for e in there}
        there = [e for e in there if choice[e] > -math.inf]
        value = {}
        for g in range(groups):
            c = sorted((choice[e] for e in there if e // size == g), reverse=True)
            if c:
                value[g] = sum(c[:best])
        kept = sorted(value, key=lambda g: (-value[g], g))[:keep]
        chosen = sorted((e for e in there if e // size in kept), key=lambda e: (-choice[e], e))[:k]
        w = [score[e] for e in chosen]
        if renormalise:
            total = math.fsum(w)
            w = [v / total if total else 0.0 for v in w]
        experts[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = [v * scale for v in w]
    return experts, weights


def adapt_reference(y, x, a, b, adapter, scales=None):
    """Returns (out [T, N], down [T, N], up [T, N]): down is scale * sum |B| of
    the first product's sums of |A x|, up that of its sums' own values."""
    out = np.array(y, dtype=np.float64)
    down, up = np.zeros(y.shape), np.zeros(y.shape)
    for t, i in enumerate(adapter):
        if 0 <= i < len(a):
            s = 1.0 if scales is None else float(scales[i])
            v = a[i] @ x[t]
            out[t] += s * (b[i] @ v)
            down[t] = abs(s) * (np.abs(b[i]) @ (np.abs(a[i]) @ np.abs(x[t])))
            up[t] = abs(s) * (np.abs(b[i]) @ np.abs(v))
    return out, down, up
