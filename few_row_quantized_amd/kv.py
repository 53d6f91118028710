"""The verify step around the quantized products, on torch device tensors:
appending the new rows' keys and values to a paged cache, with the rotation of
positions on the way or without, attention of those rows over it, also with a
prompt that the sequences share, and acceptance of the drafted tokens; routing
of rows to experts, and low-rank adapters beside a projection.

Argument marshalling only, as in :mod:`few_row_quantized_amd.qgemv`, which
offers these names: types, shapes and strides are checked (ValueError) by the
compiled module _qgemv_torch, and again by the library (:class:`QgemvError`);
the contracts stand in include/qgemv.h.

Sequence b owns rows start[b] .. start[b+1]-1 of every [T, ...] tensor (start
int32 [B+1]) and has len[b] tokens, those rows included (len int32 [B]).  Both
stay on the device: no call reads them back.
"""
from __future__ import annotations

import ctypes

import torch

from . import qgemv as _q

_TYPES = {torch.bfloat16: _q.BF16, torch.float16: _q.F16, torch.float8_e4m3fn: _q.E4M3}

_module = None


def _calls():
    """The compiled calls, bound to the library on first use."""
    global _module
    if _module is None:
        L = _q.lib()
        try:
            from . import _qgemv_torch as m
        except ImportError as e:
            raise RuntimeError(f"_qgemv_torch is not built ({e}); run `python -m few_row_quantized_amd.build`") from e
        m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.qgemv_kv_append, L.qgemv_kv_attend_workspace, L.qgemv_kv_attend, L.qgemv_verify_drafts_workspace,
            L.qgemv_verify_drafts, L.qgemv_kv_attend_shared_workspace, L.qgemv_kv_attend_shared,
            L.qgemv_kv_append_rotated, L.qgemv_route, L.qgemv_adapt_workspace, L.qgemv_adapt)), torch._C._cuda_getCurrentRawStream if torch.cuda.is_available() else None)
        _module = m
    return _module


def _allocating(stream, device):
    """`stream` as the current one: what a call allocates for itself comes from
    the stream it runs on, so that its memory is not still in use by another.
    The address 0 is the default stream, for which ExternalStream would take one
    of torch's pool that waits for nothing."""
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                  else torch.cuda.default_stream(device))
    return torch.cuda.stream(stream)


class KvCache:
    """A paged cache of keys and values: k and v [pages, page, heads, dim] of
    bfloat16, float16 or float8_e4m3fn, and table int32 [B, width], the pages
    of each sequence in order.  The last dimension is contiguous, the others may have any
    strides, the same for k and v (a permuted [pages, heads, page, dim] cache
    is one).  An 8-bit cache has k_scale and v_scale, float32 [heads].

    It holds the tensors, and no state: new pages are entered in `table` in
    place, on the stream of the calls.
    """

    def __init__(self, k, v, table, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must both be [pages, page, heads, dim], of one type and device")
        if k.dtype not in (torch.bfloat16, torch.float16, torch.float8_e4m3fn):
            raise ValueError(f"a cache of {k.dtype} is not supported")
        P, page, H, D = k.shape
        if D not in (64, 128, 256):
            raise ValueError(f"dim must be 64, 128 or 256, got {D}")
        if min(P, page, H) < 1:
            raise ValueError("k and v must not be empty")
        if k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("the last dimension of k and v must be contiguous")
        esz = k.element_size()
        strides = []
        for i, n in enumerate(k.shape[:3]):
            if n > 1 and k.stride(i) != v.stride(i):
                raise ValueError("k and v must have the same strides")
            strides.append((k.stride(i) if n > 1 else D) * esz)
        if (table.dtype != torch.int32 or table.dim() != 2 or min(table.shape) < 1
                or not table.is_contiguous() or table.device != k.device):
            raise ValueError(f"table must be a contiguous int32 [B, width] tensor on {k.device}")
        f8 = k.dtype == torch.float8_e4m3fn
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if f8 != (s is not None):
                raise ValueError(f"{name} belongs to an 8-bit cache, and such a cache needs it")
            if f8 and (s.dtype != torch.float32 or tuple(s.shape) != (H,) or not s.is_contiguous()
                       or s.device != k.device):
                raise ValueError(f"{name} must be a contiguous float32 [{H}] tensor on {k.device}")
        self.k, self.v, self.table, self.k_scale, self.v_scale = k, v, table, k_scale, v_scale
        self.device, self.dtype = k.device, k.dtype
        self.heads, self.dim, self.batch = H, D, table.shape[0]
        self._c = _q._KvCacheC(k.data_ptr(), v.data_ptr(), table.data_ptr(), _q._ptr(k_scale),
                               _q._ptr(v_scale), *strides, P, page, table.shape[1], table.shape[0], H, D,
                               _TYPES[k.dtype])
        self._ref = ctypes.byref(self._c)
        self._address = ctypes.addressof(self._c)


def append(cache: KvCache, new_k, new_v, start, len, stream=None) -> None:
    """Write the rows' keys and values, new_k and new_v [T, heads, dim] of
    float32, bfloat16 or float16, to their sequences' slots of the cache."""
    status = _calls().append(cache._address, cache.k, new_k, new_v, start, len, stream)
    if status:
        _q._check(status, "qgemv_kv_append")


def append_rotated(cache: KvCache, q, new_k, new_v, start, len, freq, position=None, axes=None,
                   interleaved: bool = False, out=None, stream=None):
    """append() with positions turned on the way: the pairs of values of the
    queries q [T, q_heads, dim] and of new_k (of one type, as new_v) by the angle
    position * freq.  freq float32 [pairs], a multiple of 8 up to dim / 2; pair
    i is the values i and pairs + i, with interleaved 2 i and 2 i + 1.  position
    int32 [A, T], the rows' positions on A axes, and axes int32 [pairs], the
    axis of each pair (the first unless given); without position a row's place
    in its sequence.  Returns the turned queries: out, else a tensor of the
    cache's type (bfloat16 for an 8-bit cache).  out may be q itself, or other
    columns of its buffer."""
    if stream is not None and out is None and cache.k.is_cuda:
        with _allocating(stream, cache.device):
            return append_rotated(cache, q, new_k, new_v, start, len, freq, position, axes, interleaved)
    r = _calls().append_rotated(cache._address, cache.k, q, new_k, new_v, start, len, freq, position, axes,
                                interleaved, out, stream)
    if type(r) is int:
        _q._check(r, "qgemv_kv_append_rotated")
    return r


def attend_workspace(cache: KvCache, M: int, q_heads: int, T: int):
    """Scratch memory for attend() calls of up to M rows a sequence and T in
    all, of any window; one for each stream that runs them."""
    need = _q._check(_q.lib().qgemv_kv_attend_workspace(cache._ref, M, q_heads, T),
                     "qgemv_kv_attend_workspace")
    return torch.empty(need, dtype=torch.uint8, device=cache.device)


def attend(cache: KvCache, q, start, len, M: int, window: int = 0, sinks: int = 0, scale=None, out=None,
           lse=None, workspace=None, stream=None):
    """Attention of the rows q [T, q_heads, dim] over their sequences' tokens,
    each row up to its own, with a window the last `window` of them and the
    first `sinks`.  M: the largest number of rows of a sequence (1..16).
    scale: dim ** -0.5 unless given.  Returns out [T, q_heads, dim]; lse, a
    float32 [T, q_heads] tensor, takes the logarithm of each row's sum."""
    if stream is not None and (out is None or workspace is None) and cache.k.is_cuda:
        with _allocating(stream, cache.device):
            return attend(cache, q, start, len, M, window, sinks, scale, out, lse, workspace)
    r = _calls().attend(cache._address, cache.k, q, start, len, M, window, sinks, scale, out, lse, workspace, stream)
    if type(r) is int:
        _q._check(r, "qgemv_kv_attend")
    return r


def attend_shared_workspace(cache: KvCache, M: int, q_heads: int, T: int):
    """Scratch memory for attend_shared() calls of up to M rows a sequence and T
    in all, of any window; one for each stream that runs them."""
    need = _q._check(_q.lib().qgemv_kv_attend_shared_workspace(cache._ref, M, q_heads, T),
                     "qgemv_kv_attend_shared_workspace")
    return torch.empty(need, dtype=torch.uint8, device=cache.device)


def attend_shared(cache: KvCache, q, start, len, M: int, shared, window: int = 0, sinks: int = 0, scale=None,
                  out=None, lse=None, workspace=None, stream=None):
    """attend() for sequences whose first tokens, `shared` of them (int32 [1] on
    the device), lie in the same pages of every sequence's table row: what they
    have in common, in whole pages, is read once for all rows."""
    if stream is not None and (out is None or workspace is None) and cache.k.is_cuda:
        with _allocating(stream, cache.device):
            return attend_shared(cache, q, start, len, M, shared, window, sinks, scale, out, lse, workspace)
    r = _calls().attend_shared(cache._address, cache.k, q, start, len, shared, M, window, sinks, scale, out, lse,
                               workspace, stream)
    if type(r) is int:
        _q._check(r, "qgemv_kv_attend_shared")
    return r


_SCORES = {"softmax": _q.SOFTMAX, "sigmoid": _q.SIGMOID}


def route(logits, k: int, score: str = "softmax", bias=None, groups: int = 1, keep: int = 1, best: int = 1,
          renormalise: bool = True, scale: float = 1.0, stream=None):
    """The k experts of each row of logits [T, E] and their weights: experts
    int32 [T, k], -1 where fewer are there, and float32 [T, k].  score "softmax"
    or "sigmoid"; bias float32 [E], added to the scores for the choice alone; of
    `groups` groups of neighbours the `keep` with the greatest sums of their
    `best` (1 or 2) greatest choices; weights over their sum unless renormalise
    is false, times scale."""
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    if stream is not None and logits.is_cuda:
        with _allocating(stream, logits.device):
            return route(logits, k, score, bias, groups, keep, best, renormalise, scale)
    r = _calls().route(logits, k, _SCORES[score], bias, groups, keep, best, renormalise, scale, stream)
    if type(r) is int:
        _q._check(r, "qgemv_route")
    return r


def adapt_workspace(a, T: int):
    """Scratch memory for adapt() calls of up to T rows with the adapters a (and
    b) or others of their rank; one for each stream that runs them."""
    need = _q._check(_q.lib().qgemv_adapt_workspace(T, a.shape[1]), "qgemv_adapt_workspace")
    return torch.empty(need, dtype=torch.uint8, device=a.device)


def adapt(y, x, a, b, adapter, scales=None, out=None, workspace=None, stream=None):
    """y + scales * B (A x) of each row's adapter: y float32 [T, N], a product
    of x [T, K]; a [n, r, K] and b [n, N, r] of x's type (bfloat16 or float16);
    adapter int32 [T], none where outside [0, n); scales float32 [n].  Returns
    out, else a new tensor; out may be y itself, or other columns of its buffer."""
    if stream is not None and (out is None or workspace is None) and y.is_cuda:
        with _allocating(stream, y.device):
            return adapt(y, x, a, b, adapter, scales, out, workspace)
    r = _calls().adapt(y, x, a, b, adapter, scales, out, workspace, stream)
    if type(r) is int:
        _q._check(r, "qgemv_adapt")
    return r


def verify_workspace(p, B: int):
    """Scratch memory for verify() calls on B sequences with p's vocabulary;
    one for each stream that runs them."""
    need = _q._check(_q.lib().qgemv_verify_drafts_workspace(B, p.shape[1]), "qgemv_verify_drafts_workspace")
    return torch.zeros(need, dtype=torch.uint8, device=p.device)


def verify(p, q, tokens, u, start, M: int, workspace=None, stream=None):
    """Accept or refuse the drafted tokens and draw the next: p [T, V] the
    target's probabilities, q [T, V] the draft model's or None, tokens int32
    [T] the token fed at each row, u float32 [T] uniform numbers.  Returns
    (out int32 [T]: each sequence's accepted drafts, its drawn token, then -1;
    count int32 [B]: how many of them are tokens)."""
    if stream is not None and p.is_cuda:
        with _allocating(stream, p.device):
            return verify(p, q, tokens, u, start, M, workspace)
    r = _calls().verify(p, q, tokens, u, start, M, workspace, stream)
    if type(r) is int:
        _q._check(r, "qgemv_verify_drafts")
    return r
