"""Binding of libsa's serving calls: attention over a paged K/V cache, the plan
of a step and the writer of new tokens.  The usual arguments take the short way
(``csrc/paged_call.cpp``), whatever else the long one, through ctypes.

Argument marshalling only, as in ``_libsa``: types, shapes and devices are
checked here, lengths, tables and sigma (device data) by the kernels, which
report through the error word (``check_error``).
"""

from __future__ import annotations

import ctypes
from ctypes import byref, c_double, c_float, c_int32, c_int64, c_void_p
from typing import NamedTuple

from . import _libsa
from ._libsa import _check, _check_err, _need, _shape

_torch = None  # set by the first call (the package imports without it)


def _get_torch():
    global _torch
    import torch
    _torch = torch
    return torch


_native = None  # paged_call.cpp's module; False: not built


def _get_native():
    global _native
    lib = _libsa._lib or _libsa.load()
    _get_torch()
    try:
        from . import _paged_call as native
    except ImportError:
        _native = False
        return False
    native.bind(*[ctypes.cast(f, c_void_p).value for f in (
        lib.swa_paged_forward, lib.sa_paged_forward, lib.sa_swa_gated_paged_forward,
        lib.sa_paged_workspace_size, lib.sa_paged_plan, lib.sa_paged_append)])
    _native = native
    return native


PAGED_AUTO, PAGED_ROWS, PAGED_TILES = 0, 1, 2
_SWA, _SA, _GATED = 0, 1, 2


class SaPagedParams(ctypes.Structure):
    """Mirror of sa_paged_params_t."""
    _fields_ = [
        ("batch", c_int32),
        ("tokens", c_int32),
        ("max_new", c_int32),
        ("num_q_heads", c_int32),
        ("num_kv_heads", c_int32),
        ("head_dim", c_int32),
        ("page_size", c_int32),
        ("num_pages", c_int32),
        ("max_pages", c_int32),
        ("window", c_int32),
        ("window_swa", c_int32),
        ("perm_rows", c_int32),
        ("perm_len", c_int32),
        ("kernel", c_int32),
        ("softmax_scale", c_float),
        ("reserved", c_int32),
        ("q_stride", c_int64),
        ("page_stride", c_int64),
        ("block_table", c_void_p),
        ("q_start", c_void_p),
        ("seq_lens", c_void_p),
        ("err", c_void_p),
    ]


class SaPagedAppendParams(ctypes.Structure):
    """Mirror of sa_paged_append_params_t."""
    _fields_ = [
        ("tokens", c_int32),
        ("num_kv_heads", c_int32),
        ("num_q_heads", c_int32),
        ("head_dim", c_int32),
        ("page_size", c_int32),
        ("num_pages", c_int32),
        ("k_stride", c_int64),
        ("v_stride", c_int64),
        ("q_stride", c_int64),
        ("page_stride", c_int64),
        ("rope_base", c_double),
        ("err", c_void_p),
    ]


class PagedPlan(NamedTuple):
    """What paged_plan wrote (int32 tensors): see paged_plan."""
    q_start: object
    seq_lens: object
    slots: object
    positions: object
    counts: object


class _On:
    """The device numbered `index` made current for the calls inside, and the
    stream they go to: the given one (made current too, so that what is
    allocated inside belongs to it), else that device's current one."""

    __slots__ = ("guards", "index")

    def __init__(self, index, stream):
        torch = _torch
        self.index = index
        self.guards = ()
        if index != torch._C._cuda_getDevice():
            self.guards = (torch.cuda.device(index),)
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=index)
            elif stream.device.index != index:
                raise ValueError(f"stream must be on cuda:{index}, got {stream.device}")
            self.guards += (torch.cuda.stream(stream),)

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return _torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _rows(t, name, dtype, ndim):
    """The shape of a contiguous tensor argument, its type and rank checked."""
    try:
        if t.dtype is dtype and t.dim() == ndim and t.is_contiguous():
            return t.shape
    except AttributeError:
        pass
    _need(t, name, dtype, ndim)  # says what is wrong


def _tokens(t, name):
    """bf16 [T, H, d] whose rows [H, d] are contiguous; returns its shape and
    the stride between tokens."""
    torch = _torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(shape)}")
    n, h, d = shape
    if t.is_contiguous():
        return shape, h * d
    st = t.stride()
    if (st[2] != 1 and d > 1) or (st[1] != d and h > 1) or (st[0] < h * d and n > 1):
        raise ValueError(f"{name} must have contiguous [heads, head_dim] rows")
    return shape, st[0] if n > 1 else h * d


def _caches(k_cache, v_cache):
    """Both caches, bf16 [pages, page_size, Hkv, d], pages contiguous and the
    same stride apart; returns their shape and that stride."""
    torch = _torch
    if not isinstance(k_cache, torch.Tensor) or not isinstance(v_cache, torch.Tensor):
        raise TypeError(f"{'v' if isinstance(k_cache, torch.Tensor) else 'k'}_cache must be a torch.Tensor")
    bf16 = torch.bfloat16
    if k_cache.dtype is not bf16 or v_cache.dtype is not bf16:
        name, t = ("v_cache", v_cache) if k_cache.dtype is bf16 else ("k_cache", k_cache)
        raise TypeError(f"{name} must be {bf16}, got {t.dtype}")
    shape = k_cache.shape
    if len(shape) != 4 or 0 in shape:
        raise ValueError(f"k_cache must be [num_pages, page_size, Hkv, d], got {tuple(shape)}")
    if v_cache.shape != shape:
        raise ValueError(f"v_cache must have shape {tuple(shape)}, got {tuple(v_cache.shape)}")
    n, ps, h, d = shape
    size = ps * h * d
    if k_cache.is_contiguous() and v_cache.is_contiguous():
        return shape, size
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        st = t.stride()
        if (st[3] != 1 and d > 1) or (st[2] != d and h > 1) or (st[1] != h * d and ps > 1) or \
                (st[0] < size and n > 1):
            raise ValueError(f"{name} must have contiguous pages")
    if n == 1:
        return shape, size
    if k_cache.stride(0) != v_cache.stride(0):
        raise ValueError("v_cache must have its pages as far apart as k_cache")
    return shape, k_cache.stride(0)


def _one_device(names, *tensors):
    """The CUDA device number that all tensors (None: not given) share; names:
    theirs, for the message."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index or index < 0:
            first = names.split()[0]
            if index < 0:
                raise ValueError(f"{first} must be a CUDA tensor")
            name = next(n for n, x in zip(names.split(), tensors) if x is t)
            raise ValueError(f"{name} must be on {tensors[0].device}, got {t.device}")
    return index


def _short(path, *args):
    """The short way of a forward call; None: the long one is needed."""
    native = _get_native() if _native is None else _native
    if not native:
        return None
    r = native.forward(path, *args)
    if r.__class__ is int:
        _check(r)
    return r


_FORWARD = "q k_cache v_cache block_table q_start seq_lens perm inv_perm gate_sa gate_swa out err"


def _forward(path, q, k_cache, v_cache, block_table, q_start, seq_lens, window, window_swa, max_new,
             softmax_scale, out, kernel, err, stream, perm=None, inv_perm=None, gate_sa=None,
             gate_swa=None):
    torch = _torch or _get_torch()
    i32 = torch.int32
    qshape, q_stride = _tokens(q, "q")
    (pages, page_size, hkv, dk), page_stride = _caches(k_cache, v_cache)
    t, hq, d = qshape
    if dk != d:
        raise ValueError(f"k_cache must have head_dim {d}, got {tuple(k_cache.shape)}")
    rows, max_pages = _rows(block_table, "block_table", i32, 2)
    b, = _rows(seq_lens, "seq_lens", i32, 1)
    if _rows(q_start, "q_start", i32, 1)[0] != b + 1:
        _shape(q_start, "q_start", (b + 1,))
    if rows != b:
        raise ValueError(f"block_table must have {b} rows, got {tuple(block_table.shape)}")
    perm_rows = perm_len = 0
    if path != _SWA:
        perm_rows, perm_len = shape = _rows(perm, "perm", i32, 2)
        if perm_rows != b and perm_rows != 1:
            raise ValueError(f"perm must have {b} rows, or one for all, got {tuple(perm.shape)}")
        if _rows(inv_perm, "inv_perm", i32, 2) != shape:
            _shape(inv_perm, "inv_perm", shape)
    if path == _GATED:
        for name, g in (("gate_sa", gate_sa), ("gate_swa", gate_swa)):
            if tuple(_rows(g, name, torch.float32, 2)) != (t, hq):
                _shape(g, name, (t, hq))
    if out is not None and _rows(out, "out", torch.bfloat16, 3) != qshape:
        _shape(out, "out", qshape)
    if err is not None:
        _check_err(err)
    index = _one_device(_FORWARD, q, k_cache, v_cache, block_table, q_start, seq_lens, perm, inv_perm,
                        gate_sa, gate_swa, out, err)
    ref = byref(SaPagedParams(b, t, int(max_new), hq, hkv, d, page_size, pages, max_pages, int(window),
                              int(window_swa), perm_rows, perm_len, int(kernel), float(softmax_scale), 0,
                              q_stride, page_stride, block_table.data_ptr(), q_start.data_ptr(),
                              seq_lens.data_ptr(), err.data_ptr() if err is not None else None))
    lib = _libsa._lib or _libsa.load()
    with _On(index, stream) as s:
        if out is None:
            out = torch.empty(qshape, dtype=torch.bfloat16, device=q.device)
        ws = lib.sa_paged_workspace_size(ref, path)
        work = torch.empty(ws, dtype=torch.uint8, device=q.device) if ws else None
        at = work.data_ptr() if ws else None
        if path == _SWA:
            st = lib.swa_paged_forward(ref, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                       out.data_ptr(), at, ws, s)
        elif path == _SA:
            st = lib.sa_paged_forward(ref, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                      perm.data_ptr(), inv_perm.data_ptr(), out.data_ptr(), at, ws, s)
        else:
            st = lib.sa_swa_gated_paged_forward(ref, q.data_ptr(), k_cache.data_ptr(),
                                                v_cache.data_ptr(), perm.data_ptr(),
                                                inv_perm.data_ptr(), gate_sa.data_ptr(),
                                                gate_swa.data_ptr(), out.data_ptr(), at, ws, s)
    if st:
        _check(st)
    return out


def swa_paged_forward(q, k_cache, v_cache, block_table, q_start, seq_lens, window: int,
                      max_new: int = 0, softmax_scale: float = 0.0, out=None,
                      kernel: int = PAGED_AUTO, err=None, stream=None):
    """Sliding-window attention of a batch's new tokens over a paged cache;
    returns out (bf16 [T, Hq, d]).

    q [T, Hq, d]: the requests' new tokens one after the other, request b's in
    rows q_start[b] .. q_start[b+1] - 1 (int32 [B+1]); tokens may be strided
    (a slice of a fused projection).  k_cache, v_cache [num_pages, page_size,
    Hkv, d] hold seq_lens[b] (int32 [B]) tokens of request b, the new ones
    included, in the pages block_table[b] (int32 [B, max_pages]) names; pages
    may be strided (kv[:, 0] and kv[:, 1]).  window >= every seq_lens[b] gives
    full causal attention.  max_new: a bound on the new tokens of any one
    request, where the caller knows one (1 when decoding).  Rows of out that
    no request has are left as they were (uninitialised if out is not given).
    """
    if stream is None:
        r = _short(_SWA, q, k_cache, v_cache, block_table, q_start, seq_lens, window, 0, max_new, softmax_scale,
                   out, kernel, err, None, None, None, None)
        if r is not None:
            return r
    return _forward(_SWA, q, k_cache, v_cache, block_table, q_start, seq_lens, window, 0, max_new,
                    softmax_scale, out, kernel, err, stream)


def sa_paged_forward(q, k_cache, v_cache, block_table, q_start, seq_lens, perm, inv_perm,
                     window: int, max_new: int = 0, softmax_scale: float = 0.0, out=None,
                     kernel: int = PAGED_AUTO, err=None, stream=None):
    """Causal Stochastic Attention of a batch's new tokens over a paged cache.

    perm and inv_perm (int32 [B, n], or [1, n] shared by all requests): sigma
    of each request, drawn for the n tokens it may reach at most, and its
    inverse (sa_inverse_perm).  The rows equal those of sa_forward(causal=True)
    on the whole sequence.  The rest as in swa_paged_forward.
    """
    if stream is None:
        r = _short(_SA, q, k_cache, v_cache, block_table, q_start, seq_lens, window, 0, max_new, softmax_scale,
                   out, kernel, err, perm, inv_perm, None, None)
        if r is not None:
            return r
    return _forward(_SA, q, k_cache, v_cache, block_table, q_start, seq_lens, window, 0, max_new,
                    softmax_scale, out, kernel, err, stream, perm, inv_perm)


def sa_swa_gated_paged_forward(q, k_cache, v_cache, block_table, q_start, seq_lens, perm, inv_perm,
                               gate_sa, gate_swa, window: int, window_swa: int = 0,
                               max_new: int = 0, softmax_scale: float = 0.0, out=None,
                               kernel: int = PAGED_AUTO, err=None, stream=None):
    """sigmoid(gate_sa) * SA + sigmoid(gate_swa) * SWA over a paged cache; the
    gate logits (fp32 [T, Hq]) are the new tokens'."""
    if stream is None:
        r = _short(_GATED, q, k_cache, v_cache, block_table, q_start, seq_lens, window, window_swa, max_new,
                   softmax_scale, out, kernel, err, perm, inv_perm, gate_sa, gate_swa)
        if r is not None:
            return r
    return _forward(_GATED, q, k_cache, v_cache, block_table, q_start, seq_lens, window, window_swa,
                    max_new, softmax_scale, out, kernel, err, stream, perm, inv_perm, gate_sa, gate_swa)


def paged_plan(new_lens, cached_lens, block_table, free_pages, num_free, page_size: int,
               num_pages: int, max_tokens: int, q_start=None, seq_lens=None, slots=None,
               positions=None, counts=None, err=None, stream=None) -> PagedPlan:
    """Plan of one step on the device: request b has cached_lens[b] tokens in
    its pages and brings new_lens[b] more (int32 [B]).  Pages are taken from
    the top of free_pages (int32 [F], the first num_free[0] of them free) and
    written into block_table (int32 [B, max_pages], in place); returns
    q_start [B+1], seq_lens [B], slots and positions [max_tokens] (-1 past the
    last token) and counts [3] = new tokens, pages taken, pages left.  If the
    step does not fit, nothing is planned and the error word says so."""
    if stream is q_start is seq_lens is slots is positions is counts is None:
        native = _get_native() if _native is None else _native
        r = native.plan(new_lens, cached_lens, block_table, free_pages, num_free, page_size, num_pages,
                        max_tokens, err) if native else None
        if r is not None:
            if r.__class__ is int:
                _check(r)
            return PagedPlan._make(r)
    torch = _torch or _get_torch()
    i32 = torch.int32
    b, = _rows(new_lens, "new_lens", i32, 1)
    if _rows(cached_lens, "cached_lens", i32, 1)[0] != b:
        _shape(cached_lens, "cached_lens", (b,))
    rows, max_pages = _rows(block_table, "block_table", i32, 2)
    if rows != b:
        raise ValueError(f"block_table must have {b} rows, got {tuple(block_table.shape)}")
    free_capacity, = _rows(free_pages, "free_pages", i32, 1)
    if _rows(num_free, "num_free", i32, 1)[0] != 1:
        _shape(num_free, "num_free", (1,))
    n = int(max_tokens)
    if n < 0:
        raise ValueError("max_tokens must be >= 0")
    if err is not None:
        _check_err(err)
    outs = (q_start, seq_lens, slots, positions, counts)
    sizes = (b + 1, b, n, n, 3)
    for i, t in enumerate(outs):
        if t is not None and _rows(t, PagedPlan._fields[i], i32, 1)[0] != sizes[i]:
            _shape(t, PagedPlan._fields[i], (sizes[i],))
    index = _one_device("new_lens cached_lens block_table free_pages num_free err q_start seq_lens slots "
                        "positions counts", new_lens, cached_lens, block_table, free_pages, num_free, err, *outs)
    lib = _libsa._lib or _libsa.load()
    with _On(index, stream) as s:
        if any(t is None for t in outs):  # what is not given, cut from one allocation
            new = torch.empty(sum(sizes), dtype=i32, device=new_lens.device).split_with_sizes(sizes)
            outs = [x if t is None else t for t, x in zip(outs, new)]
        st = lib.sa_paged_plan(new_lens.data_ptr(), cached_lens.data_ptr(), b, block_table.data_ptr(),
                               max_pages, free_pages.data_ptr(), free_capacity, num_free.data_ptr(),
                               int(page_size), int(num_pages), n, *[t.data_ptr() for t in outs],
                               err.data_ptr() if err is not None else None, s)
    if st:
        _check(st)
    return PagedPlan(*outs)


def paged_append(k, v, k_cache, v_cache, slots, positions=None, rope_base: float = 0.0, q=None,
                 q_out=None, err=None, stream=None):
    """New tokens' k and v (bf16 [T, Hkv, d], tokens may be strided) into the
    rows slots (int32 [T], page * page_size + row; -1: padding, skipped) of
    the caches.  With rope_base > 1 the keys are rotated by positions (int32
    [T]) as rope_ does, and q (bf16 [T, Hq, d]) is rotated into q_out, which
    is returned; otherwise None is."""
    if stream is None:
        native = _get_native() if _native is None else _native
        r = native.append(k, v, k_cache, v_cache, slots, positions, rope_base, q, q_out, err) if native else None
        if r is not None:
            if r is True:
                return None
            if r.__class__ is int:
                _check(r)
            return r
    torch = _torch or _get_torch()
    (t, hkv, d), ks = _tokens(k, "k")
    vshape, vs = _tokens(v, "v")
    if vshape != k.shape:
        _shape(v, "v", k.shape)
    (pages, page_size, hc, dc), page_stride = _caches(k_cache, v_cache)
    if hc != hkv or dc != d:
        raise ValueError(f"k_cache must be [num_pages, page_size, {hkv}, {d}], got {tuple(k_cache.shape)}")
    if _rows(slots, "slots", torch.int32, 1)[0] != t:
        _shape(slots, "slots", (t,))
    rope_base = float(rope_base)
    rope = rope_base != 0.0
    if positions is not None:
        if _rows(positions, "positions", torch.int32, 1)[0] != t:
            _shape(positions, "positions", (t,))
    elif rope:
        raise ValueError("positions are needed with rope_base")
    hq = qs = 0
    if q is not None:
        if not rope:
            raise ValueError("q is rotated only: it needs rope_base")
        qshape, qs = _tokens(q, "q")
        hq = qshape[1]
        if qshape[0] != t or qshape[2] != d:
            _shape(q, "q", (t, hq, d))
        if q_out is not None and _rows(q_out, "q_out", torch.bfloat16, 3) != qshape:
            _shape(q_out, "q_out", qshape)
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    if err is not None:
        _check_err(err)
    index = _one_device("k v k_cache v_cache slots positions q q_out err", k, v, k_cache, v_cache, slots,
                        positions, q, q_out, err)
    ref = byref(SaPagedAppendParams(t, hkv, hq, d, page_size, pages, ks, vs, qs, page_stride, rope_base,
                                    err.data_ptr() if err is not None else None))
    lib = _libsa._lib or _libsa.load()
    with _On(index, stream) as s:
        if q is not None and q_out is None:
            q_out = torch.empty((t, hq, d), dtype=torch.bfloat16, device=k.device)
        st = lib.sa_paged_append(ref, k.data_ptr(), v.data_ptr(), q.data_ptr() if q is not None else None,
                                 slots.data_ptr(), positions.data_ptr() if rope else None,
                                 k_cache.data_ptr(), v_cache.data_ptr(),
                                 q_out.data_ptr() if q is not None else None, s)
    if st:
        _check(st)
    return q_out
