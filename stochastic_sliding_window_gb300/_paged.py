"""ctypes binding of libsa's serving calls: attention over a paged K/V cache,
the plan of a step and the writer of new tokens.

Argument marshalling only, as in ``_libsa``: types, shapes and devices are
checked here, lengths, tables and sigma (device data) by the kernels, which
report through the error word (``check_error``).
"""

from __future__ import annotations

import ctypes
from ctypes import byref, c_double, c_float, c_int32, c_int64, c_void_p
from typing import NamedTuple

from . import _libsa
from ._libsa import _check, _check_err, _need, _on_device, _shape

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
    """The device of `t` made current for the calls inside, and the stream
    they go to: the given one (made current too, so that what is allocated
    inside belongs to it), else that device's current one."""

    __slots__ = ("guards", "device")

    def __init__(self, t, stream):
        import torch
        self.device = t.device
        self.guards = []
        if t.device.index != torch.cuda.current_device():
            self.guards.append(torch.cuda.device(t.device))
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=t.device)
            elif stream.device != t.device:
                raise ValueError(f"stream must be on {t.device}, got {stream.device}")
            self.guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        import torch
        for g in self.guards:
            g.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _tokens(t, name):
    """bf16 [T, H, d] whose rows [H, d] are contiguous; returns the stride
    between tokens."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(t.shape)}")
    n, h, d = t.shape
    st = t.stride()
    if n * h * d and ((st[2] != 1 and d > 1) or (st[1] != d and h > 1) or (st[0] < h * d and n > 1)):
        raise ValueError(f"{name} must have contiguous [heads, head_dim] rows")
    return st[0] if n > 1 else h * d


def _caches(k_cache, v_cache):
    """Both caches, bf16 [pages, page_size, Hkv, d], pages contiguous and the
    same stride apart; returns that stride."""
    import torch
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
        if t.dim() != 4 or 0 in t.shape:
            raise ValueError(f"{name} must be [num_pages, page_size, Hkv, d], got {tuple(t.shape)}")
    if k_cache.shape != v_cache.shape:
        raise ValueError(f"v_cache must have shape {tuple(k_cache.shape)}, got {tuple(v_cache.shape)}")
    n, ps, h, d = k_cache.shape
    size = ps * h * d
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        st = t.stride()
        if (st[3] != 1 and d > 1) or (st[2] != d and h > 1) or (st[1] != h * d and ps > 1) or \
                (st[0] < size and n > 1):
            raise ValueError(f"{name} must have contiguous pages")
    if n == 1:
        return size
    if k_cache.stride(0) != v_cache.stride(0):
        raise ValueError("v_cache must have its pages as far apart as k_cache")
    return k_cache.stride(0)


def _forward(path, q, k_cache, v_cache, block_table, q_start, seq_lens, window, window_swa, max_new,
             softmax_scale, out, kernel, err, stream, perm=None, inv_perm=None, gate_sa=None,
             gate_swa=None):
    import torch
    q_stride = _tokens(q, "q")
    page_stride = _caches(k_cache, v_cache)
    t, hq, d = q.shape
    pages, page_size, hkv, dk = k_cache.shape
    if dk != d:
        raise ValueError(f"k_cache must have head_dim {d}, got {tuple(k_cache.shape)}")
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(q_start, "q_start", torch.int32, 1)
    b = seq_lens.shape[0]
    _shape(q_start, "q_start", (b + 1,))
    if block_table.shape[0] != b:
        raise ValueError(f"block_table must have {b} rows, got {tuple(block_table.shape)}")
    named = [("k_cache", k_cache), ("v_cache", v_cache), ("block_table", block_table),
             ("q_start", q_start), ("seq_lens", seq_lens), ("err", err)]
    perm_rows = perm_len = 0
    if path != _SWA:
        _need(perm, "perm", torch.int32, 2)
        _need(inv_perm, "inv_perm", torch.int32, 2)
        perm_rows, perm_len = perm.shape
        if perm_rows != b and perm_rows != 1:
            raise ValueError(f"perm must have {b} rows, or one for all, got {tuple(perm.shape)}")
        _shape(inv_perm, "inv_perm", perm.shape)
        named += [("perm", perm), ("inv_perm", inv_perm)]
    if path == _GATED:
        for name, g in (("gate_sa", gate_sa), ("gate_swa", gate_swa)):
            _need(g, name, torch.float32, 2)
            _shape(g, name, (t, hq))
            named.append((name, g))
    if out is not None:
        _need(out, "out", torch.bfloat16, 3)
        _shape(out, "out", q.shape)
        named.append(("out", out))
    _check_err(err)
    _on_device(q, "q", named)
    prm = SaPagedParams(b, t, int(max_new), hq, hkv, d, page_size, pages, block_table.shape[1],
                        int(window), int(window_swa), perm_rows, perm_len, int(kernel),
                        float(softmax_scale), 0, q_stride, page_stride, block_table.data_ptr(),
                        q_start.data_ptr(), seq_lens.data_ptr(),
                        err.data_ptr() if err is not None else None)
    ref = byref(prm)
    lib = _libsa.load()
    with _On(q, stream) as s:
        if out is None:
            out = torch.empty((t, hq, d), dtype=torch.bfloat16, device=q.device)
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
    return _forward(_SA, q, k_cache, v_cache, block_table, q_start, seq_lens, window, 0, max_new,
                    softmax_scale, out, kernel, err, stream, perm, inv_perm)


def sa_swa_gated_paged_forward(q, k_cache, v_cache, block_table, q_start, seq_lens, perm, inv_perm,
                               gate_sa, gate_swa, window: int, window_swa: int = 0,
                               max_new: int = 0, softmax_scale: float = 0.0, out=None,
                               kernel: int = PAGED_AUTO, err=None, stream=None):
    """sigmoid(gate_sa) * SA + sigmoid(gate_swa) * SWA over a paged cache; the
    gate logits (fp32 [T, Hq]) are the new tokens'."""
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
    import torch
    for name, t in (("new_lens", new_lens), ("cached_lens", cached_lens),
                    ("free_pages", free_pages), ("num_free", num_free)):
        _need(t, name, torch.int32, 1)
    _need(block_table, "block_table", torch.int32, 2)
    b = new_lens.shape[0]
    _shape(cached_lens, "cached_lens", (b,))
    if block_table.shape[0] != b:
        raise ValueError(f"block_table must have {b} rows, got {tuple(block_table.shape)}")
    _shape(num_free, "num_free", (1,))
    n = int(max_tokens)
    if n < 0:
        raise ValueError("max_tokens must be >= 0")
    _check_err(err)
    given = [("q_start", q_start, b + 1), ("seq_lens", seq_lens, b), ("slots", slots, n),
             ("positions", positions, n), ("counts", counts, 3)]
    for name, t, size in given:
        if t is not None:
            _need(t, name, torch.int32, 1)
            _shape(t, name, (size,))
    _on_device(new_lens, "new_lens", [("cached_lens", cached_lens), ("block_table", block_table),
                                      ("free_pages", free_pages), ("num_free", num_free),
                                      ("err", err)] + [(x[0], x[1]) for x in given])
    ptr = lambda t: t.data_ptr() if t.numel() else None
    with _On(new_lens, stream) as s:
        outs = [torch.empty(size, dtype=torch.int32, device=new_lens.device) if t is None else t
                for _, t, size in given]
        st = _libsa.load().sa_paged_plan(
            ptr(new_lens), ptr(cached_lens), b, ptr(block_table), block_table.shape[1],
            ptr(free_pages), free_pages.shape[0], ptr(num_free), int(page_size), int(num_pages), n,
            *[ptr(t) for t in outs], err.data_ptr() if err is not None else None, s)
    _check(st)
    return PagedPlan(*outs)


def paged_append(k, v, k_cache, v_cache, slots, positions=None, rope_base: float = 0.0, q=None,
                 q_out=None, err=None, stream=None):
    """New tokens' k and v (bf16 [T, Hkv, d], tokens may be strided) into the
    rows slots (int32 [T], page * page_size + row; -1: padding, skipped) of
    the caches.  With rope_base > 1 the keys are rotated by positions (int32
    [T]) as rope_ does, and q (bf16 [T, Hq, d]) is rotated into q_out, which
    is returned; otherwise None is."""
    import torch
    ks, vs = _tokens(k, "k"), _tokens(v, "v")
    page_stride = _caches(k_cache, v_cache)
    t, hkv, d = k.shape
    _shape(v, "v", k.shape)
    pages, page_size, hc, dc = k_cache.shape
    if (hc, dc) != (hkv, d):
        raise ValueError(f"k_cache must be [num_pages, page_size, {hkv}, {d}], got {tuple(k_cache.shape)}")
    _need(slots, "slots", torch.int32, 1)
    _shape(slots, "slots", (t,))
    rope = float(rope_base) != 0.0
    if positions is not None:
        _need(positions, "positions", torch.int32, 1)
        _shape(positions, "positions", (t,))
    elif rope:
        raise ValueError("positions are needed with rope_base")
    hq = qs = 0
    if q is not None:
        if not rope:
            raise ValueError("q is rotated only: it needs rope_base")
        qs = _tokens(q, "q")
        hq = q.shape[1]
        _shape(q, "q", (t, hq, d))
        if q_out is not None:
            _need(q_out, "q_out", torch.bfloat16, 3)
            _shape(q_out, "q_out", q.shape)
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    _check_err(err)
    _on_device(k, "k", [("v", v), ("k_cache", k_cache), ("v_cache", v_cache), ("slots", slots),
                        ("positions", positions), ("q", q), ("q_out", q_out), ("err", err)])
    prm = SaPagedAppendParams(t, hkv, hq, d, page_size, pages, ks, vs, qs, page_stride,
                              float(rope_base), err.data_ptr() if err is not None else None)
    with _On(k, stream) as s:
        if q is not None and q_out is None:
            q_out = torch.empty((t, hq, d), dtype=torch.bfloat16, device=k.device)
        st = _libsa.load().sa_paged_append(
            byref(prm), k.data_ptr(), v.data_ptr(), q.data_ptr() if q is not None else None,
            slots.data_ptr(), positions.data_ptr() if rope else None, k_cache.data_ptr(),
            v_cache.data_ptr(), q_out.data_ptr() if q is not None else None, s)
    _check(st)
    return q_out
