"""The verify step around the quantized products, on torch device tensors:
appending the new rows' keys and values to a paged cache, attention of those
rows over it, and acceptance of the drafted tokens.

Argument marshalling only, as in :mod:`few_row_quantized_amd.qgemv`, which
offers these names: types, shapes and strides are checked here (ValueError)
and again by the library (:class:`QgemvError`); the contracts stand in
include/qgemv.h.

Sequence b owns rows start[b] .. start[b+1]-1 of every [T, ...] tensor (start
int32 [B+1]) and has len[b] tokens, those rows included (len int32 [B]).  Both
stay on the device: no call reads them back.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import qgemv as _q

_TYPES = {torch.float32: _q.F32, torch.bfloat16: _q.BF16, torch.float16: _q.F16,
          torch.float8_e4m3fn: _q.E4M3}


def _strides(name: str, t, dim: int):
    """Row and head strides of a [T, heads, dim] operand, in elements.  A
    dimension of one element has no stride of its own: it gets a packed one."""
    if t.dim() != 3 or t.shape[2] != dim or t.stride(2) != 1:
        raise ValueError(f"{name} must be [T, heads, {dim}] with a contiguous last dimension")
    T, heads, _ = t.shape
    head = t.stride(1) if heads > 1 else dim
    return t.stride(0) if T > 1 else heads * head, head


def _index(name: str, t, n: int, device):
    if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous int32 [{n}] tensor on {device}")
    return t.data_ptr()


def _on(device, stream) -> Optional[int]:
    """The raw stream of a call on `device`, which has to be the current one."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on the GPU, not on {device}")
    if device.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {device}, the current device is {torch.cuda.current_device()}")
    return _q._stream(stream)


def _new(shape, dtype, device, stream, fill=None):
    """A tensor for a call on `stream`, allocated there, so that its memory is
    not still in use by another stream."""
    if stream is not None and device.type == "cuda":
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        with torch.cuda.stream(stream):
            return _new(shape, dtype, device, None, fill)
    t = torch.empty(shape, dtype=dtype, device=device)
    return t if fill is None else t.fill_(fill)


def _work(workspace, need: int, device, stream, zeroed: bool):
    if workspace is None:
        return _new((need,), torch.uint8, device, stream, 0 if zeroed else None)
    if workspace.dtype != torch.uint8 or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace


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


def append(cache: KvCache, new_k, new_v, start, len, stream=None) -> None:
    """Write the rows' keys and values, new_k and new_v [T, heads, dim] of
    float32, bfloat16 or float16, to their sequences' slots of the cache."""
    dev, D = cache.device, cache.dim
    if new_k.dtype != new_v.dtype or new_k.dtype not in _TYPES or new_k.dtype == torch.float8_e4m3fn:
        raise ValueError(f"new_k and new_v must be float32, bfloat16 or float16, got {new_k.dtype}, {new_v.dtype}")
    if new_k.shape != new_v.shape or new_k.shape[1] != cache.heads or new_k.device != dev or new_v.device != dev:
        raise ValueError(f"new_k and new_v must be [T, {cache.heads}, {D}] on {dev}")
    k_row, k_head = _strides("new_k", new_k, D)
    v_row, v_head = _strides("new_v", new_v, D)
    s, n = _index("start", start, cache.batch + 1, dev), _index("len", len, cache.batch, dev)
    T = new_k.shape[0]
    if T == 0:
        return
    _q._check(_q.lib().qgemv_kv_append(cache._ref, new_k.data_ptr(), k_row, k_head, new_v.data_ptr(),
                                       v_row, v_head, _TYPES[new_k.dtype], s, n, T, _on(dev, stream)),
              "qgemv_kv_append")


def attend_workspace(cache: KvCache, M: int, q_heads: int, T: int):
    """Scratch memory for attend() calls of this size; one for each stream
    that runs them."""
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
    dev, D = cache.device, cache.dim
    if q.dtype not in (torch.bfloat16, torch.float16) or cache.dtype not in (q.dtype, torch.float8_e4m3fn):
        raise ValueError(f"q of {q.dtype} over a cache of {cache.dtype} is not supported")
    if q.device != dev:
        raise ValueError(f"q must be on {dev}")
    q_row, q_head = _strides("q", q, D)
    T, heads, _ = q.shape
    s, n = _index("start", start, cache.batch + 1, dev), _index("len", len, cache.batch, dev)
    if out is None:
        out = _new((T, heads, D), q.dtype, dev, stream)
        o_row, o_head = heads * D, D
    else:
        if out.dtype != q.dtype or out.shape != q.shape or out.device != dev:
            raise ValueError("out must have q's type, shape and device")
        o_row, o_head = _strides("out", out, D)
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (T, heads) or not lse.is_contiguous()
                            or lse.device != dev):
        raise ValueError(f"lse must be a contiguous float32 [{T}, {heads}] tensor on {dev}")
    L = _q.lib()
    if workspace is None:
        need = _q._check(L.qgemv_kv_attend_workspace(cache._ref, M, heads, T), "qgemv_kv_attend_workspace")
        workspace = _work(None, need, dev, stream, False)
    else:
        _work(workspace, 0, dev, stream, False)
    if T == 0:
        return out
    _q._check(L.qgemv_kv_attend(cache._ref, q.data_ptr(), q_row, q_head, out.data_ptr(), o_row, o_head,
                                _TYPES[q.dtype], None if lse is None else lse.data_ptr(), s, n, T, M, heads,
                                window, sinks, D ** -0.5 if scale is None else scale,
                                workspace.data_ptr(), workspace.numel(), _on(dev, stream)),
              "qgemv_kv_attend")
    return out


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
    dev = p.device
    if p.dtype not in _TYPES or p.dtype == torch.float8_e4m3fn or p.dim() != 2 or p.shape[1] < 1:
        raise ValueError("p must be a float32, bfloat16 or float16 [T, V] tensor")
    T, V = p.shape
    for name, t in (("p", p), ("q", q)):
        if t is not None and (t.shape != p.shape or t.dtype != p.dtype or t.device != dev
                              or (V > 1 and t.stride(1) != 1)):
            raise ValueError(f"{name} must be a {p.dtype} [{T}, {V}] tensor on {dev} with contiguous rows")
    B = start.shape[0] - 1
    if B < 1:
        raise ValueError("start must have at least two entries")
    s = _index("start", start, B + 1, dev)
    k = _index("tokens", tokens, T, dev)
    if u.dtype != torch.float32 or u.shape != (T,) or not u.is_contiguous() or u.device != dev:
        raise ValueError(f"u must be a contiguous float32 [{T}] tensor on {dev}")
    out = _new((T,), torch.int32, dev, stream)
    count = _new((B,), torch.int32, dev, stream)
    if T == 0:
        return out, count.zero_()
    L = _q.lib()
    if workspace is None:
        need = _q._check(L.qgemv_verify_drafts_workspace(B, V), "qgemv_verify_drafts_workspace")
        workspace = _work(None, need, dev, stream, True)
    else:
        _work(workspace, 0, dev, stream, True)
    _q._check(L.qgemv_verify_drafts(p.data_ptr(), p.stride(0) if T > 1 else V, None if q is None else q.data_ptr(),
                                    0 if q is None else q.stride(0) if T > 1 else V, _TYPES[p.dtype], k,
                                    u.data_ptr(), s, out.data_ptr(), count.data_ptr(), B, T, M, V,
                                    workspace.data_ptr(), workspace.numel(), _on(dev, stream)),
              "qgemv_verify_drafts")
    return out, count
