"""Serving calls on the host: refusals before anything is launched, and the
oracle of the paged attention against the whole-sequence oracle."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import oracle
import stochastic_sliding_window_gb300 as sa

B, T, HQ, HKV, D, PAGES, PAGE, WIDTH, N = 2, 5, 8, 2, 64, 6, 16, 3, 40


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _i(*shape):
    return _t(*shape, dtype=torch.int32)


def _good():
    return dict(q=_t(T, HQ, D), k_cache=_t(PAGES, PAGE, HKV, D), v_cache=_t(PAGES, PAGE, HKV, D),
                block_table=_i(B, WIDTH), q_start=_i(B + 1), seq_lens=_i(B), perm=_i(B, N),
                inv_perm=_i(B, N), gate_sa=_t(T, HQ, dtype=torch.float32),
                gate_swa=_t(T, HQ, dtype=torch.float32), window=16)


def _call(path, a):
    base = ["q", "k_cache", "v_cache", "block_table", "q_start", "seq_lens", "window", "out", "err"]
    more = {"swa": [], "sa": ["perm", "inv_perm"],
            "gated": ["perm", "inv_perm", "gate_sa", "gate_swa"]}[path]
    fn = {"swa": sa.swa_paged_forward, "sa": sa.sa_paged_forward, "gated": sa.sa_swa_gated_paged_forward}[path]
    return fn(**{k: a[k] for k in base + more if k in a})


BAD = [
    ("q", _t(T, HQ * D), ValueError), ("q", _t(T, HQ, D).float(), TypeError),
    ("q", _t(T, D, HQ).transpose(1, 2), ValueError), ("q", None, TypeError),
    ("k_cache", _t(PAGES, PAGE, HKV, 128), ValueError), ("k_cache", _t(PAGES, HKV, PAGE, D).transpose(1, 2), ValueError),
    ("v_cache", _t(PAGES + 1, PAGE, HKV, D), ValueError), ("v_cache", _t(PAGES, 2, PAGE, HKV, D)[:, 0], ValueError),
    ("k_cache", _t(0, PAGE, HKV, D), ValueError),
    ("block_table", _i(B + 1, WIDTH), ValueError), ("block_table", _i(B, WIDTH).long(), TypeError),
    ("q_start", _i(B), ValueError), ("seq_lens", _i(B, 1), ValueError),
    ("perm", _i(3, N), ValueError), ("inv_perm", _i(B, N - 1), ValueError),
    ("gate_sa", _t(T, HKV, dtype=torch.float32), ValueError), ("gate_swa", _t(T, HQ), TypeError),
    ("out", _t(T - 1, HQ, D), ValueError), ("err", _t(1, dtype=torch.int64), TypeError),
]


@pytest.mark.parametrize("field,bad,kind", BAD, ids=[f"{i}-{x[0]}" for i, x in enumerate(BAD)])
@pytest.mark.parametrize("path", ["swa", "sa", "gated"])
def test_forward_refuses_malformed_arguments(path, field, bad, kind):
    if (path == "swa" and field in ("perm", "inv_perm")) or (path != "gated" and field.startswith("gate")):
        pytest.skip("argument not taken")
    a = _good()
    a[field] = bad
    with pytest.raises(kind):
        _call(path, a)


@pytest.mark.parametrize("path", ["swa", "sa", "gated"])
def test_well_formed_cpu_tensors_are_refused(path):
    with pytest.raises(ValueError, match="CUDA"):
        _call(path, _good())


def test_strided_queries_and_pages_are_taken_as_far_as_the_device_check():
    a = _good()
    a["q"] = _t(T, HQ + 2 * HKV, D)[:, :HQ]
    kv = _t(PAGES, 2, PAGE, HKV, D)
    a["k_cache"], a["v_cache"] = kv[:, 0], kv[:, 1]
    with pytest.raises(ValueError, match="CUDA"):
        _call("swa", a)


def _params(**kw):
    base = dict(batch=2, tokens=4, max_new=0, num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16,
                num_pages=10, max_pages=4, window=8, window_swa=0, perm_rows=2, perm_len=50, kernel=0,
                softmax_scale=0.0, reserved=0, q_stride=0, page_stride=0, block_table=0x1000,
                q_start=0x2000, seq_lens=0x3000, err=0x4000)
    base.update(kw)
    return sa.SaPagedParams(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 1), (dict(tokens=-1), 1), (dict(num_kv_heads=3), 1), (dict(head_dim=96), 2),
    (dict(page_size=0), 1), (dict(num_pages=1 << 28), 2), (dict(max_pages=0), 1), (dict(window=0), 1),
    (dict(kernel=3), 1), (dict(kernel=-1), 1), (dict(q_stride=500), 1), (dict(q_stride=516), 1),
    (dict(page_stride=2040), 1), (dict(tokens=1 << 29), 2), (dict(block_table=None), 1),
    (dict(q_start=None), 1), (dict(seq_lens=None), 1),
])
def test_c_call_refuses_bad_sizes(kw, status):
    lib = sa.load()
    prm = _params(**kw)
    p = lambda i: ctypes.c_void_p(0x100000 * i)  # never dereferenced
    assert lib.swa_paged_forward(ctypes.byref(prm), p(1), p(2), p(3), p(4), p(5), 1 << 30, None) == status
    assert lib.sa_last_error_message().decode() != ""


def test_c_call_refuses_bad_pointers_and_sigma():
    lib = sa.load()
    ref = ctypes.byref
    p = lambda i: ctypes.c_void_p(0x100000 * i)
    good = _params()
    bad = sa.SA_ERR_INVALID_ARG
    assert lib.swa_paged_forward(None, p(1), p(2), p(3), p(4), None, 0, None) == bad
    assert lib.swa_paged_forward(ref(good), None, p(2), p(3), p(4), None, 0, None) == bad
    assert lib.swa_paged_forward(ref(good), ctypes.c_void_p(0x100008), p(2), p(3), p(4), None, 0, None) == bad
    assert lib.swa_paged_forward(ref(good), p(1), p(2), p(3), p(1), None, 0, None) == bad
    assert lib.sa_paged_forward(ref(good), p(1), p(2), p(3), None, p(6), p(4), None, 0, None) == bad
    assert lib.sa_paged_forward(ref(_params(perm_rows=3)), p(1), p(2), p(3), p(5), p(6), p(4), None, 0, None) == bad
    assert lib.sa_paged_forward(ref(_params(kernel=2)), p(1), p(2), p(3), p(5), p(6), p(4), None, 0,
                                None) == sa.SA_ERR_UNSUPPORTED
    assert lib.sa_swa_gated_paged_forward(ref(good), p(1), p(2), p(3), p(5), p(6), None, p(7), p(4), None, 0,
                                          None) == bad
    # no tokens: nothing to do, whatever the pointers
    assert lib.swa_paged_forward(ref(_params(tokens=0)), None, None, None, None, None, 0, None) == sa.SA_OK
    for path in range(-1, 4):
        assert lib.sa_paged_workspace_size(ref(_params(batch=0)), path) == 0


def test_plan_refusals():
    ok = dict(new_lens=_i(B), cached_lens=_i(B), block_table=_i(B, WIDTH), free_pages=_i(9), num_free=_i(1),
              page_size=16, num_pages=10, max_tokens=8)
    for bad in (dict(new_lens=_i(B).long()), dict(cached_lens=_i(B + 1)), dict(block_table=_i(1, WIDTH)),
                dict(num_free=_i(2)), dict(max_tokens=-1), dict(slots=_i(7)), dict(q_start=_i(B))):
        with pytest.raises((TypeError, ValueError)):
            sa.paged_plan(**{**ok, **bad})
    with pytest.raises(ValueError, match="CUDA"):
        sa.paged_plan(**ok)
    lib = sa.load()
    p = [ctypes.c_void_p(0x1000 * i) for i in range(1, 20)]
    call = lambda b=2, mp=3, cap=9, page=16, pages=10, tok=8, seq=p[6]: lib.sa_paged_plan(
        p[0], p[1], b, p[2], mp, p[3], cap, p[4], page, pages, tok, p[5], seq, p[7], p[8], p[9], p[10], None)
    for kw in (dict(b=0), dict(mp=0), dict(cap=-1), dict(page=0), dict(pages=0), dict(tok=-1), dict(seq=p[1])):
        assert call(**kw) == sa.SA_ERR_INVALID_ARG
    assert call(pages=1 << 28) == sa.SA_ERR_UNSUPPORTED


def test_append_refusals():
    ok = dict(k=_t(T, HKV, D), v=_t(T, HKV, D), k_cache=_t(PAGES, PAGE, HKV, D), v_cache=_t(PAGES, PAGE, HKV, D),
              slots=_i(T), positions=_i(T), rope_base=10.0, q=_t(T, HQ, D))
    for bad in (dict(v=_t(T, HKV, 32)), dict(k_cache=_t(PAGES, PAGE, HKV + 1, D), v_cache=_t(PAGES, PAGE, HKV + 1, D)),
                dict(slots=_i(T + 1)), dict(positions=None), dict(rope_base=0.0), dict(q=_t(T + 1, HQ, D)),
                dict(q=None, q_out=_t(T, HQ, D)), dict(q_out=_t(T, HQ, 32))):
        with pytest.raises((TypeError, ValueError)):
            sa.paged_append(**{**ok, **bad})
    with pytest.raises(ValueError, match="CUDA"):
        sa.paged_append(**ok)
    lib = sa.load()
    p = lambda i: ctypes.c_void_p(0x100000 * i)
    prm = lambda **kw: ctypes.byref(sa.SaPagedAppendParams(**{**dict(
        tokens=4, num_kv_heads=2, num_q_heads=8, head_dim=64, page_size=16, num_pages=10, rope_base=10.0), **kw}))
    call = lambda q=p(3), qo=p(8), kc=p(6), **kw: lib.sa_paged_append(prm(**kw), p(1), p(2), q, p(4), p(5), kc, p(7),
                                                                     qo, None)
    for kw in (dict(tokens=-1), dict(num_kv_heads=0), dict(head_dim=63), dict(head_dim=258), dict(page_size=0),
               dict(rope_base=0.5), dict(rope_base=float("nan")), dict(rope_base=0.0), dict(num_q_heads=0),
               dict(k_stride=100), dict(page_stride=8), dict(qo=p(3)), dict(kc=p(7)), dict(qo=None)):
        assert call(**kw) == sa.SA_ERR_INVALID_ARG, kw
    assert call(num_pages=1 << 28) == sa.SA_ERR_UNSUPPORTED
    assert call(tokens=0) == sa.SA_OK


@pytest.mark.parametrize("path", ["swa", "sa", "gated"])
def test_paged_oracle_equals_the_whole_sequence_oracle(path):
    """Rows fed in two chunks over shuffled pages are the rows of the
    whole-sequence oracle (causal)."""
    rng = np.random.default_rng(1)
    n, hq, hkv, d, page = 30, 4, 2, 8, 4
    q, k, v = (rng.standard_normal((1, n, h, d)) for h in (hq, hkv, hkv))
    ga, gw = rng.standard_normal((1, n, hq)), rng.standard_normal((1, n, hq))
    perm = oracle.make_perm(5, 0, 0, n)[None]
    whole = {"swa": lambda: oracle.swa_forward(q, k, v, 7),
             "sa": lambda: oracle.sa_forward(q, k, v, perm, 6, True),
             "gated": lambda: oracle.gated_forward(q, k, v, perm, ga, gw, 6, 7, True)}[path]()
    pages = rng.permutation(12)
    kc, vc = np.full((12, page, hkv, d), np.nan), np.full((12, page, hkv, d), np.nan)
    j = np.arange(n)
    kc[pages[j // page], j % page], vc[pages[j // page], j % page] = k[0], v[0]
    for lo, hi in ((0, 13), (13, 30)):
        got, spread = oracle.paged_attention(path, q[0, lo:hi], kc, vc, pages[None, :], [0, hi - lo], [hi],
                                             7 if path == "swa" else 6, 7, perm, ga[0, lo:hi], gw[0, lo:hi])
        assert np.abs(got - whole[0, lo:hi]).max() < 1e-12
        assert (spread >= np.abs(got) - 1e-12).all()


def test_plan_oracle_counts_pages():
    p = oracle.paged_plan([5, 0, 3], [3, 4, 0], [[2, -1, -1], [3, -1, -1], [-1, -1, -1]], [7, 8, 9], 3, 4, 10)
    assert p["block_table"].tolist() == [[2, 9, -1], [3, -1, -1], [8, -1, -1]]
    assert p["slots"].tolist() == [11, 36, 37, 38, 39, 32, 33, 34, -1, -1]
    assert p["counts"].tolist() == [8, 2, 1]
    assert oracle.paged_plan([5], [3], [[2, -1]], [7], 0, 4, 10) is None
