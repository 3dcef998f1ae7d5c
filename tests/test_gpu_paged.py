"""Serving calls on the GPU against the fp64 oracle: the paged attention of
the three paths, the plan of a step, the writer of new tokens, and a run of
them together against the whole-sequence calls."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import stochastic_sliding_window_gb300 as sa
from paged_helpers import Batch, bf16, err_word, i32

pytestmark = pytest.mark.gpu

ALL = 1 << 30

# new tokens, tokens in all, Hq, Hkv, d, page
SHAPES = {
    "one_token": ([1], [1], 4, 1, 64, 16),
    "decode_gqa": ([1, 1, 1, 1, 1], [300, 1, 17, 16, 129], 8, 2, 128, 16),
    "decode_mha": ([1, 1, 1], [97, 33, 200], 3, 3, 64, 7),
    "decode_g5": ([1, 1], [77, 150], 10, 2, 128, 1),
    "decode_g20": ([1, 1], [64, 90], 20, 1, 64, 33),
    "decode_g16": ([1, 0, 1], [64, 5, 90], 32, 2, 128, 8),
    "verify": ([5, 1, 3, 8], [60, 40, 3, 256], 8, 2, 128, 16),
    "verify_mha": ([4, 17, 1], [100, 17, 65], 2, 2, 64, 32),
    "chunks": ([33, 1, 0, 20], [70, 300, 12, 20], 8, 4, 64, 48),
    "empty_first": ([0, 0, 3], [9, 0, 50], 4, 4, 128, 5),
}


@pytest.mark.parametrize("window", [1, 2, 31, 128, ALL])
@pytest.mark.parametrize("shape", SHAPES)
def test_swa_rows(shape, window):
    new, total, hq, hkv, d, page = SHAPES[shape]
    b = Batch(new, total, hq, hkv, d, page, seed=window % 97 + len(shape))
    err = err_word()
    out = b.run("swa", window, kernel=sa.PAGED_ROWS, max_new=max(new), err=err)
    assert sa.check_error(err) == sa.SA_OK
    b.check(out, "swa", window, what=shape)


TILE_SHAPES = {
    "one_row": ([1], [1], 1, 1, 64, 16),
    "chunk_gqa": ([200, 1, 0, 65], [700, 300, 5, 65], 8, 2, 128, 16),
    "chunk_mha": ([300, 257, 20], [300, 1000, 21], 2, 2, 64, 7),
    "chunk_g5": ([90, 52], [130, 77], 10, 2, 128, 33),
    "chunk_g64": ([9, 4], [40, 300], 64, 1, 64, 1),
    "long": ([130], [9000], 8, 2, 128, 64),
    "ragged": ([70, 3, 129, 1, 64, 500], [71, 3, 640, 2000, 64, 501], 8, 4, 64, 100),
}


@pytest.mark.parametrize("window", [1, 100, 129, 1000, ALL])
@pytest.mark.parametrize("shape", TILE_SHAPES)
def test_swa_tiles(shape, window):
    new, total, hq, hkv, d, page = TILE_SHAPES[shape]
    b = Batch(new, total, hq, hkv, d, page, seed=window % 97 + len(shape))
    err = err_word()
    out = b.run("swa", window, kernel=sa.PAGED_TILES, err=err)
    assert sa.check_error(err) == sa.SA_OK
    b.check(out, "swa", window, weight_bits=8, what=shape)
    assert torch.equal(out, b.run("swa", window, kernel=sa.PAGED_TILES, max_new=max(new)))


@pytest.mark.parametrize("path", ["swa", "gated"])
@pytest.mark.parametrize("shape", TILE_SHAPES)
def test_auto_mixes_both_kernels(path, shape):
    """Requests of few and of many new tokens in one call."""
    new, total, hq, hkv, d, page = TILE_SHAPES[shape]
    b = Batch(new, total, hq, hkv, d, page, seed=len(shape), perm_len=max(total), behind=3)
    out = torch.full((b.t + 3, hq, d), 2.0, dtype=torch.bfloat16, device="cuda")
    err = err_word()
    b.run(path, 90, 200, out=out, err=err)
    assert sa.check_error(err) == sa.SA_OK
    b.check(out, path, 90, 200, weight_bits=8, what=shape)
    assert (out[b.t:] == 2.0).all()


SA_TILE_SHAPES = {
    "one_request": ([300], [700], 8, 2, 128, 16, 700),
    "mha": ([300, 257, 20], [300, 1000, 21], 2, 2, 64, 7, 1500),
    "g5": ([190, 152], [230, 177], 10, 2, 128, 33, 1000),
    "g64": ([60, 40, 1], [60, 300, 80], 64, 1, 64, 1, 300),
    "long": ([600], [9000], 4, 1, 128, 64, 9001),
    "ragged": ([70, 3, 129, 1, 64, 500, 0], [71, 3, 640, 2000, 64, 501, 30], 8, 4, 64, 100, 2500),
    "all_at_once": ([2000], [2000], 4, 2, 64, 64, 2000),
}


@pytest.mark.parametrize("window", [1, 33, 128, 700])
@pytest.mark.parametrize("shape", SA_TILE_SHAPES)
@pytest.mark.parametrize("path", ["sa", "gated"])
def test_sa_tiles(path, shape, window):
    """Chunks whose SA path goes to the tiles (and, among them, requests that
    do not)."""
    new, total, hq, hkv, d, page, cap = SA_TILE_SHAPES[shape]
    b = Batch(new, total, hq, hkv, d, page, seed=window + len(shape), perm_len=cap, behind=2,
              shared_perm=window == 33, stride_q=64, pair_pages=window == 128)
    out = torch.full((b.t + 2, hq, d), 2.0, dtype=torch.bfloat16, device="cuda")
    err = err_word()
    b.run(path, window, 77, out=out, err=err, max_new=max(new))
    assert sa.check_error(err) == sa.SA_OK
    b.check(out, path, window, 77, weight_bits=8, what=f"{path} {shape}")
    assert (out[b.t:] == 2.0).all()
    again = b.run(path, window, 77)
    assert torch.equal(out[:b.t], again[:b.t])


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 2, 128), (3, 3, 64), (10, 2, 128), (32, 2, 64)])
@pytest.mark.parametrize("path", ["sa", "gated"])
def test_sa_of_requests_far_apart_and_close_in_one_call(path, hq, hkv, d):
    """New tokens that are all of a long request, some of one and few of one:
    their windows share much, little and nothing."""
    b = Batch([1500, 300, 40, 1], [1600, 1400, 700, 90], hq, hkv, d, 32, seed=hq, perm_len=3001, behind=1)
    out = torch.full((b.t + 1, hq, d), 2.0, dtype=torch.bfloat16, device="cuda")
    err = err_word()
    b.run(path, 128, 100, out=out, err=err, max_new=1500)
    assert sa.check_error(err) == sa.SA_OK
    b.check(out, path, 128, 100, weight_bits=8, what=path)
    assert (out[b.t:] == 2.0).all()
    assert torch.equal(b.run(path, 128, 100)[:b.t], out[:b.t])


def test_members_with_bad_sigma_and_pages():
    """As for tiles: bad pages' keys are left out and reported, rows that a bad
    sigma does not name are left as they were."""
    b = Batch([200], [1500], 4, 2, 128, 16, seed=2, perm_len=6000)
    good = b.run("sa", 300).clone()
    table = b.args[3].clone()
    table[0, 3:9] = -5
    table[0, 60:] = 1 << 30
    args = list(b.args)
    args[3] = table
    err = err_word()
    out = sa.sa_paged_forward(*args, b.perm_d, b.inv_d, window=300, err=err)
    assert sa.check_error(err) == sa.SA_ERR_BAD_PERM and torch.isfinite(out).all()
    perm = b.perm_d.clone()
    perm[0, perm[0] == 1400] = 7  # token 1400 named nowhere
    err.zero_()
    out = torch.full_like(good, 3.0)
    sa.sa_paged_forward(*b.args, perm, b.inv_d, window=300, out=out, err=err)
    assert sa.check_error(err) == sa.SA_ERR_BAD_PERM
    assert (out == 3.0).all(-1).all(-1).sum() == 1


def test_sa_tiles_with_bad_sigma_and_pages():
    b = Batch([200], [500], 4, 2, 64, 16, seed=2, perm_len=600)
    good = b.run("sa", 64).clone()
    table = b.args[3].clone()
    table[0, 3] = -5
    args = list(b.args)
    args[3] = table
    err = err_word()
    out = sa.sa_paged_forward(*args, b.perm_d, b.inv_d, window=64, err=err)
    assert sa.check_error(err) == sa.SA_ERR_BAD_PERM and torch.isfinite(out).all()
    for bad in (-1, 600, 1 << 30):  # an entry out of range: rows may be missing, nothing is read out of bounds
        perm = b.perm_d.clone()
        perm[0, 17] = bad
        err = err_word()
        sa.sa_paged_forward(*b.args, perm, b.inv_d, window=64, err=err)
        assert sa.check_error(err) == sa.SA_ERR_BAD_PERM
    perm = b.perm_d.clone()
    perm[0, perm[0].long() == 450] = 10  # one new token twice missing, another token twice
    err = err_word()
    out = sa.sa_paged_forward(*b.args, perm, b.inv_d, window=64, err=err,
                              out=torch.full_like(good, 5.0))
    assert sa.check_error(err) == sa.SA_ERR_BAD_PERM
    assert (out[150] == 5.0).all()  # the missing token's row is left
    err = err_word()
    assert torch.equal(sa.sa_paged_forward(*b.args, b.perm_d, b.inv_d, window=64, err=err), good)
    assert sa.check_error(err) == sa.SA_OK


def test_sa_tiles_of_requests_that_claim_the_same_rows():
    """q_start that goes back: more long requests than rows allow."""
    b = Batch([200] * 6, [200] * 6, 4, 2, 64, 16, seed=2, perm_len=200)
    starts = i32([0, 200, 0, 200, 0, 200, 0])
    args = list(b.args)
    args[0], args[4] = b.q[:200], starts
    for path in ("sa", "gated"):
        err = err_word()
        b.args = tuple(args)
        b.gate_sa, b.gate_swa = b.gate_sa[:200].contiguous(), b.gate_swa[:200].contiguous()
        b.run(path, 64, 64, err=err)
        assert sa.check_error(err) == sa.SA_ERR_BAD_PERM


def test_tiles_whose_reference_rises():
    """Scores that grow along the keys by far more than 2^8 a chunk: O is
    rescaled, and the first chunks' weights vanish."""
    b = Batch([100], [1200], 4, 1, 128, 16, seed=3)
    ramp = torch.linspace(0.05, 6.0, b.num_pages * 16, device="cuda").view(-1, 16, 1, 1)
    b.q = b.args[0].abs()
    order = torch.empty(b.num_pages, dtype=torch.long, device="cuda")
    rest = np.setdiff1d(np.arange(b.num_pages), b.table[0])
    order[torch.from_numpy(np.concatenate([b.table[0][b.table[0] >= 0], rest])).cuda()] = \
        torch.arange(b.num_pages, device="cuda")
    b.k = (b.k.abs() * ramp[order]).to(torch.bfloat16)
    b.args = (b.q, b.k) + b.args[2:]
    for kernel in (sa.PAGED_ROWS, sa.PAGED_TILES):
        out = b.run("swa", ALL, kernel=kernel)
        b.check(out, "swa", ALL, weight_bits=8, what=str(kernel))


def test_tiles_with_bad_pages_and_lengths():
    b = Batch([70, 80], [300, 400], 4, 2, 64, 16, seed=2)
    table = b.table.copy()
    table[0, 5] = -1
    table[0, 18] = b.num_pages
    args = list(b.args)
    args[3] = i32(table)
    b.args = tuple(args)
    err = err_word()
    out = b.run("swa", ALL, kernel=sa.PAGED_TILES, err=err)
    assert sa.check_error(err) == sa.SA_ERR_BAD_PERM
    assert torch.isfinite(out).all()
    # the bad pages' keys are left out, as if the request had not had them
    f = lambda x: x.float().cpu().numpy().astype(np.float64)
    k, v = f(b.k), f(b.v)
    j = np.array([x for x in range(300) if x // 16 not in (5, 18)])
    kk, vv = k[table[0, j // 16], j % 16], v[table[0, j // 16], j % 16]
    for i in (0, 33, 69):
        live = j <= 230 + i
        s = np.einsum("hgd,jhd->hgj", f(b.q)[i].reshape(2, 2, 64), kk[live]) / 8
        p = np.exp(s - s.max(-1, keepdims=True))
        y = np.einsum("hgj,jhd->hgd", p / p.sum(-1, keepdims=True), vv[live]).reshape(4, 64)
        assert np.abs(f(out)[i] - y).max() < 0.03
    err = err_word()
    args[5] = i32([300, 79])
    b.args = tuple(args)
    out.fill_(6.0)
    b.run("swa", ALL, kernel=sa.PAGED_TILES, err=err, out=out)
    assert (out[70:] == 6.0).all() and sa.check_error(err) == sa.SA_ERR_BAD_PERM


def test_tile_waits_give_up_within_their_bound():
    """A wait limit far below a chunk's time: the call returns with the
    timeout bit, the context stays usable."""
    b = Batch([300], [3000], 8, 2, 128, 1, seed=1)  # pages of one token: the slowest loads
    err = err_word()
    sa.set_wait_limit(1)
    try:
        b.run("swa", ALL, kernel=sa.PAGED_TILES, err=err)
        assert sa.check_error(err) == sa.SA_ERR_TIMEOUT
    finally:
        sa.set_wait_limit(0)
    err = err_word()
    out = b.run("swa", ALL, kernel=sa.PAGED_TILES, err=err)
    assert sa.check_error(err) == sa.SA_OK
    b.check(out, "swa", ALL, weight_bits=8)


@pytest.mark.parametrize("window", [1, 16, 129])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("path", ["sa", "gated"])
def test_sa_and_gated_rows(path, shape, window):
    new, total, hq, hkv, d, page = SHAPES[shape]
    b = Batch(new, total, hq, hkv, d, page, seed=window + 5, perm_len=max(total) + window % 3,
              shared_perm=window == 16)
    err = err_word()
    out = b.run(path, window, 40, kernel=sa.PAGED_ROWS, err=err)
    assert sa.check_error(err) == sa.SA_OK
    b.check(out, path, window, 40, what=f"{path} {shape}")


@pytest.mark.parametrize("path", ["swa", "sa", "gated"])
def test_strides_rows_behind_and_scale(path):
    """q as a slice of a wider array, K and V interleaved by page, rows of q
    and out behind the last request, a scale of the caller's."""
    b = Batch([1, 4, 2], [50, 90, 2], 8, 2, 64, 16, seed=3, behind=5, stride_q=64, pair_pages=True,
              perm_len=100)
    out = torch.full((b.t + 5, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    err = err_word()
    got = b.run(path, 24, 9, out=out, softmax_scale=0.3, err=err)
    assert got is out and sa.check_error(err) == sa.SA_OK
    b.check(out, path, 24, 9, scale=0.3, what=path)
    assert (out[b.t:] == 7.0).all()


@pytest.mark.parametrize("path", ["swa", "sa", "gated"])
def test_many_splits_agree_with_the_oracle_and_repeat_bitwise(path):
    """One long request: its units are cut over many workers."""
    n = 5000
    b = Batch([1], [n], 8, 2, 128, 64, seed=11, perm_len=n)
    window = 3001
    got = b.run(path, window, ALL)
    b.check(got, path, window, ALL, what=path)
    for _ in range(3):
        assert torch.equal(got, b.run(path, window, ALL))


def test_peaked_scores_and_large_values():
    b = Batch([1, 3], [400, 77], 8, 2, 128, 16, seed=5, spread=12.0)
    b.check(b.run("swa", ALL), "swa", ALL, what="peaked")


def test_snapped_runs_of_many_units():
    """More units than four per worker: runs end at unit ends."""
    new = [900, 1, 700, 401]
    total = [950, 333, 700, 1000]
    b = Batch(new, total, 16, 16, 64, 32, seed=8, perm_len=1000)
    b.check(b.run("sa", 20, kernel=sa.PAGED_ROWS), "sa", 20, what="sa")
    b.check(b.run("gated", 20, 13, kernel=sa.PAGED_ROWS), "gated", 20, 13, what="gated")
    b.check(b.run("swa", 13, kernel=sa.PAGED_ROWS), "swa", 13, what="swa")


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements with the request in its last pages."""
    page, hkv, d, num = 64, 8, 128, 40000
    assert num * page * hkv * d > 2 ** 31
    b = Batch([2], [200], 16, hkv, d, page, seed=21, perm_len=200)
    table = b.table + (num - b.num_pages) * (b.table >= 0)
    k = torch.empty(num, page, hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    k[num - b.num_pages:], v[num - b.num_pages:] = b.k, b.v
    args = (b.q, k, v, i32(table)) + b.args[4:]
    b.check(sa.swa_paged_forward(*args, window=90), "swa", 90, what="swa")
    b.check(sa.sa_paged_forward(*args, b.perm_d, b.inv_d, window=90), "sa", 90, what="sa")
    # and the writer: the last row of the last page
    slots = i32([num * page - 1])
    row = bf16(np.random.default_rng(0).standard_normal((1, hkv, d)))
    sa.paged_append(row, -row, k, v, slots)
    assert torch.equal(k[-1, -1], row[0]) and torch.equal(v[-1, -1], -row[0])
    del k, v
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ device checks

@pytest.mark.parametrize("path", ["swa", "sa", "gated"])
@pytest.mark.parametrize("bad_page", [-1, -(1 << 31), 1 << 30])
def test_bad_pages_are_reported_and_not_read(path, bad_page):
    b = Batch([1, 2], [60, 60], 4, 2, 64, 16, seed=2, perm_len=64)
    table = b.table.copy()
    table[0, 1] = bad_page
    args = list(b.args)
    args[3] = i32(table)
    b.args = tuple(args)
    err = err_word()
    out = b.run(path, 64, ALL, err=err)
    assert sa.check_error(err) == sa.SA_ERR_BAD_PERM
    assert torch.isfinite(out).all()
    # the other request is untouched by it
    want, _ = b.want(path, 64, ALL)
    assert np.abs(out[1:].float().cpu().numpy() - want[1:]).max() < 0.05


@pytest.mark.parametrize("path", ["swa", "sa", "gated"])
def test_a_request_whose_pages_are_all_bad_gives_zero_rows(path):
    b = Batch([1], [20], 4, 2, 64, 16, seed=2, perm_len=20)
    args = list(b.args)
    args[3] = torch.full_like(args[3], b.num_pages)
    b.args = tuple(args)
    err = err_word()
    out = b.run(path, 9, 9, err=err)
    assert sa.check_error(err) == sa.SA_ERR_BAD_PERM
    assert (out == 0).all()


@pytest.mark.parametrize("path", ["swa", "sa", "gated"])
@pytest.mark.parametrize("what", ["short", "long", "rows", "negative", "max_new"])
def test_bad_lengths_leave_their_rows(path, what):
    b = Batch([1, 3, 1], [20, 30, 25], 4, 2, 64, 16, seed=4, perm_len=40)
    total, starts, kw = list(b.total), list(b.q_start), {}
    bad = 1
    if what == "short":
        total[1] = 2
    elif what == "long":
        total[1] = 3 * 16 + 1  # one more than three table entries hold
    elif what == "rows":
        starts[3], bad = b.t + 1, 2
    elif what == "negative":
        total[1] = -5
    else:
        kw["max_new"] = 2
    args = list(b.args)
    args[4], args[5] = i32(starts), i32(total)
    b.args = tuple(args)
    out = torch.full((b.t, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    err = err_word()
    b.run(path, 9, 9, out=out, err=err, **kw)
    assert sa.check_error(err) == sa.SA_ERR_BAD_PERM
    rows = slice(b.q_start[bad], b.q_start[bad + 1])
    assert (out[rows] == 9.0).all()
    good = np.ones(b.t, bool)
    good[rows] = False
    want, _ = b.want(path, 9, 9)
    assert np.abs(out.float().cpu().numpy() - want)[good].max() < 0.05


@pytest.mark.parametrize("entry", [-1, 64, 1 << 30])
@pytest.mark.parametrize("which", ["perm", "inv", "short"])
def test_bad_sigma_is_reported(which, entry):
    b = Batch([2], [60], 4, 2, 64, 16, seed=2, perm_len=64)
    if which == "perm":
        b.perm_d[0] = entry
    elif which == "inv":
        b.inv_d[0, 58:60] = entry
    else:  # a request longer than sigma
        b.perm_d, b.inv_d = b.perm_d[:, :59].contiguous(), b.inv_d[:, :59].contiguous()
    err = err_word()
    out = b.run("sa", 16, err=err, out=torch.full((2, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda"))
    assert sa.check_error(err) == sa.SA_ERR_BAD_PERM
    if which != "short":
        assert (out == 0).all()  # nothing attended
    else:
        assert (out == 3.0).all()


# ------------------------------------------------------------------ plan

@pytest.mark.parametrize("batch,page,longest", [(1, 1, 3), (1, 16, 100), (37, 16, 40), (513, 8, 33),
                                                (1200, 5, 20), (3, 64, 5000)])
def test_plan(batch, page, longest):
    rng = np.random.default_rng(batch)
    new = rng.integers(0, longest + 1, batch)
    cached = rng.integers(0, longest + 1, batch)
    width = -(-2 * longest // page) + 1
    owned = -(-cached // page)
    ids = rng.permutation(int(owned.sum()) + batch * width)
    table = np.full((batch, width), -1)
    at = 0
    for b in range(batch):
        table[b, :owned[b]] = ids[at:at + owned[b]]
        at += owned[b]
    free = np.concatenate([ids[at:], [-7, -7]])
    cap = int(new.sum()) + 9
    want = oracle.paged_plan(new, cached, table, free, len(free) - 2, page, cap)
    table_d = i32(table)
    err = err_word()
    plan = sa.paged_plan(i32(new), i32(cached), table_d, i32(free), i32([len(free) - 2]), page,
                         len(ids), cap, err=err)
    assert sa.check_error(err) == sa.SA_OK
    for name, w in want.items():
        got = table_d if name == "block_table" else getattr(plan, name)
        assert np.array_equal(got.cpu().numpy(), w), name


@pytest.mark.parametrize("what", ["pages", "tokens", "table", "new", "cached", "free"])
def test_plan_that_does_not_fit_changes_nothing(what):
    new, cached, table = [5, 9, 2], [3, 0, 20], np.array([[4, -1, -1], [-1, -1, -1], [1, 2, 3]])
    free, num, cap = [9, 8, 7, 6], 3, 20
    if what == "pages":
        num = 1
    elif what == "tokens":
        cap = 15
    elif what == "table":
        new[2] = 5
    elif what == "new":
        new[0] = -1
    elif what == "cached":
        cached[1] = -2
    else:
        num = 5  # more than the list holds
    table_d, err = i32(table), err_word()
    plan = sa.paged_plan(i32(new), i32(cached), table_d, i32(free), i32([num]), 8, 16, cap, err=err)
    assert sa.check_error(err) == sa.SA_ERR_BAD_PERM
    assert np.array_equal(table_d.cpu().numpy(), table)
    assert (plan.q_start == 0).all() and plan.seq_lens.tolist() == cached
    assert (plan.slots == -1).all() and (plan.positions == -1).all()
    assert plan.counts.tolist() == [0, 0, num]


def test_plan_reports_bad_page_ids():
    table_d, err = i32([[99, -1]]), err_word()
    plan = sa.paged_plan(i32([3]), i32([6]), table_d, i32([5, 40]), i32([2]), 8, 16, 4, err=err)
    assert sa.check_error(err) == sa.SA_ERR_BAD_PERM
    assert plan.slots.tolist() == [-1, -1, -1, -1] and plan.positions.tolist() == [6, 7, 8, -1]


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("d,hkv,hq,page,shift", [(128, 8, 32, 16, 0), (64, 2, 8, 7, 0), (6, 1, 3, 4, 0),
                                                 (128, 2, 4, 16, 1), (256, 1, 2, 5, 0), (72, 3, 3, 9, 3)])
@pytest.mark.parametrize("rope", [False, True])
def test_append(d, hkv, hq, page, shift, rope):
    """Rows at any alignment (shift: elements off a 16-byte boundary); the
    rows that no slot names keep what they held."""
    rng = np.random.default_rng(d + hkv)
    t, pages = 301, 80
    width = (hq + 2 * hkv) * d
    flat = bf16(rng.standard_normal(t * width + shift))
    qkv = flat[shift:].view(t, hq + 2 * hkv, d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    kc = torch.full((pages, page, hkv, d), 5.0, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    slots = np.full(t, -1)
    live = rng.permutation(t)[:min(t - 3, pages * page - 1)]
    slots[live] = rng.permutation(pages * page)[:len(live)]
    positions = rng.integers(0, 1 << 31, t)
    positions[:8] = [0, 1, 2, 3, 1000, 32767, 262143, (1 << 31) - 1]
    err = err_word()
    out = torch.full((t, hq, d), 4.0, dtype=torch.bfloat16, device="cuda")
    got = sa.paged_append(k, v, kc, vc, i32(slots), i32(positions), rope_base=10000.0 if rope else 0.0,
                          q=q if rope else None, q_out=out if rope else None, err=err)
    assert sa.check_error(err) == sa.SA_OK
    f = lambda x: x.float().cpu().numpy().astype(np.float64)
    kf, vf = f(kc).reshape(-1, hkv, d), f(vc).reshape(-1, hkv, d)
    named = slots[live]
    assert np.array_equal(vf[named], f(v)[live])
    other = np.setdiff1d(np.arange(pages * page), named)
    assert (kf[other] == 5.0).all() and (vf[other] == 5.0).all()
    if not rope:
        assert got is None and np.array_equal(kf[named], f(k)[live])
        return

    def near(have, x, pos):
        # The frequency is held to 2^-53 of itself in turns (so the angle to
        # 2 pi 2^-53 p / (2 pi) = p 2^-53 radians, at most 2^-22, and the
        # oracle's own angle likewise), the angle to a step of 2^-32 turns and
        # fp32 rounding of it (2^-24 of at most pi), sine and cosine to 2^-23
        # each; two products and a sum of size |x| in fp32; one bf16 rounding.
        want = oracle.rotate_at(x, pos, 10000.0)
        half = d // 2
        size = np.hypot(x[..., :half], x[..., half:])
        size = np.concatenate([size, size], -1)
        rel = 2 * 2.0 ** -22 + 2 * np.pi * 2.0 ** -32 + np.pi * 2.0 ** -24 + 2 * 2.0 ** -23 + 4 * 2.0 ** -24
        bar = rel * size
        bar = bar + 2.0 ** -8 * (np.abs(want) + bar)
        assert (np.abs(have - want) <= bar).all(), float((np.abs(have - want) / bar).max())

    near(kf[named], f(k)[live], positions[live])
    assert got is out
    near(f(out)[live], f(q)[live], positions[live])
    rest = np.setdiff1d(np.arange(t), live)
    assert (f(out)[rest] == 4.0).all()


@pytest.mark.parametrize("d,hkv,hq,t", [(80, 2, 5, 700), (16, 8, 32, 2000), (256, 40, 4, 31), (48, 1, 1, 3000),
                                        (64, 70, 140, 10), (128, 1, 1, 1300), (96, 3, 7, 1), (64, 8, 32, 1000)])
def test_append_of_many_shapes(d, hkv, hq, t):
    """Heads that the threads of a block take in one round or in several, with
    threads over, and one or several tokens to a block.  (Tolerance as in
    test_append, at positions below 2^15, where the frequencies' rounding is
    less than the angle's.)"""
    rng = np.random.default_rng(d + t)
    qkv = bf16(rng.standard_normal((t, hq + 2 * hkv, d)))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    kc = torch.zeros(t // 16 + 1, 16, hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    slots, positions = rng.permutation(kc.shape[0] * 16)[:t], rng.integers(0, 1 << 15, t)
    err = err_word()
    out = sa.paged_append(k, v, kc, vc, i32(slots), i32(positions), rope_base=500.0, q=q, err=err)
    assert sa.check_error(err) == sa.SA_OK
    f = lambda x: x.float().cpu().numpy().astype(np.float64)
    for have, x in ((f(kc).reshape(-1, hkv, d)[slots], f(k)), (f(out), f(q))):
        want = oracle.rotate_at(x, positions, 500.0)
        size = np.hypot(x[..., :d // 2], x[..., d // 2:])
        rel = 2 * 2.0 ** -22 + 2 * np.pi * 2.0 ** -32 + np.pi * 2.0 ** -24 + 2 * 2.0 ** -23 + 4 * 2.0 ** -24
        bar = rel * np.concatenate([size, size], -1)
        bar = bar + 2.0 ** -8 * (np.abs(want) + bar)
        assert (np.abs(have - want) <= bar).all()
    assert np.array_equal(f(vc).reshape(-1, hkv, d)[slots], f(v))


def test_append_agrees_with_rope_on_a_sequence():
    """Positions 0 .. n-1: the same rotation as rope_, up to one rounding step
    of bf16 where the two angles' last bits differ."""
    n, h, d = 700, 4, 128
    x = bf16(np.random.default_rng(0).standard_normal((1, n, h, d)))
    kc = torch.zeros(n, 1, h, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    sa.paged_append(x[0], x[0], kc, vc, at, at, rope_base=500000.0)
    y = sa.rope_(x.clone(), base=500000.0)[0].float()
    off = (kc[:, 0].float() - y).abs()
    # both within 2^-8 |y| + 2^-20 |x| of the exact rotation
    assert (off <= 2 * (2.0 ** -8 * y.abs() + 2.0 ** -20 * 8)).all()


@pytest.mark.parametrize("slot,position", [(64, 0), (-2, 0), (1 << 30, 0), (3, -1)])
def test_append_reports_bad_slots(slot, position):
    k = bf16(np.ones((2, 1, 64)))
    kc = torch.zeros(4, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    err = err_word()
    sa.paged_append(k, k, kc, vc, i32([7, slot]), i32([0, position]), rope_base=100.0, err=err)
    assert sa.check_error(err) == sa.SA_ERR_BAD_PERM
    assert int((kc != 0).any(-1).sum()) == 1 and (vc[0, 7] == 1).all()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("path", ["swa", "sa", "gated"])
def test_steps_of_a_serving_loop_equal_the_whole_sequence_call(path):
    """Three sequences fed in chunks and single tokens through plan, append
    and attention, against the whole-sequence call on each."""
    rng = np.random.default_rng(17)
    hq, hkv, d, page, n, window, wswa = 8, 2, 128, 16, 260, 32, 24
    batch, pages, width = 3, 60, 20
    q, k, v = (bf16(rng.standard_normal((batch, n, h, d))) for h in (hq, hkv, hkv))
    ga, gw = (torch.from_numpy(rng.standard_normal((batch, n, hq)).astype(np.float32)).cuda() for _ in range(2))
    perm = torch.from_numpy(sa.make_perms(3, 0, batch, n)).cuda()
    inv = sa.sa_inverse_perm(perm)
    qr, kr = sa.rope_(q.clone(), 1e4), sa.rope_(k.clone(), 1e4)
    if path == "swa":
        whole = sa.swa_forward(qr, kr, v, wswa)
    elif path == "sa":
        whole = sa.sa_forward(qr, kr, v, perm, window)
    else:
        whole = sa.sa_swa_gated_forward(qr, kr, v, perm, ga, gw, window, wswa)
    kc = torch.full((pages, page, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda()
    num_free = i32([pages])
    cached = i32([0] * batch)
    steps = [[100, 1, 0], [1, 37, 16], [1, 1, 1], [60, 1, 17], [1, 0, 31], [97, 220, 195]]
    got = torch.empty_like(q)
    at = [0] * batch
    err = err_word()
    for step in steps:
        cap = sum(step) + 3
        pick = [(b, at[b] + i) for b in range(batch) for i in range(step[b])]
        rows = lambda x: torch.cat([torch.stack([x[b, i] for b, i in pick]),
                                    torch.full((3,) + x.shape[2:], float("nan"), dtype=x.dtype, device="cuda")])
        plan = sa.paged_plan(i32(step), cached, table, free, num_free, page, pages, cap, err=err)
        qn = sa.paged_append(rows(k), rows(v), kc, vc, plan.slots, plan.positions, rope_base=1e4, q=rows(q),
                             err=err)
        where = (qn, kc, vc, table, plan.q_start, plan.seq_lens)
        if path == "swa":
            y = sa.swa_paged_forward(*where, window=wswa, max_new=max(step), err=err)
        elif path == "sa":
            y = sa.sa_paged_forward(*where, perm, inv, window=window, max_new=max(step), err=err)
        else:
            y = sa.sa_swa_gated_paged_forward(*where, perm, inv, rows(ga), rows(gw), window=window,
                                              window_swa=wswa, max_new=max(step), err=err)
        for r, (b, i) in enumerate(pick):
            got[b, i] = y[r]
        cached, num_free = plan.seq_lens, plan.counts[2:].clone()
        at = [a + s for a, s in zip(at, step)]
    assert at == [n] * batch and sa.check_error(err) == sa.SA_OK
    # Both sides: their own roundings of the keys' rotation (half a step of
    # bf16 where the angle's last bit differs), of the weights and of the
    # result (twice for the gated whole-sequence call); the kernels' parity
    # bounds of the whole-sequence tests, once for each side.
    off = (got.float() - whole.float())
    assert off.abs().max().item() <= 2 * 2e-2
    assert (off.norm() / whole.float().norm()).item() <= 2 * 5e-3


@pytest.mark.parametrize("path", ["swa", "sa", "gated"])
def test_captured_graph_reads_the_lengths_of_its_replay(path):
    a = Batch([1, 1, 2], [40, 90, 33], 8, 2, 64, 16, seed=6, perm_len=100)
    b = Batch([2, 1, 1], [41, 90, 21], 8, 2, 64, 16, seed=9, perm_len=100)
    out = torch.empty(4, 8, 64, dtype=torch.bfloat16, device="cuda")
    width = max(a.args[3].shape[1], b.args[3].shape[1])
    pages = max(a.num_pages, b.num_pages)
    static = Batch.__new__(Batch)
    static.__dict__.update(a.__dict__)
    grow = lambda x: torch.cat([x, torch.zeros(pages - x.shape[0], *x.shape[1:], dtype=x.dtype, device="cuda")])
    tab = lambda x: torch.nn.functional.pad(x, (0, width - x.shape[1]), value=-1).contiguous()
    whole = lambda s: [s.q, grow(s.k), grow(s.v), tab(s.args[3]), s.args[4], s.args[5]]
    static.args = tuple(t.clone() for t in whole(a))
    for name in ("perm_d", "inv_d", "gate_sa", "gate_swa"):
        setattr(static, name, getattr(a, name).clone())
    err = err_word()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        static.run(path, 20, 30, out=out, err=err, max_new=2)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static.run(path, 20, 30, out=out, err=err, max_new=2)
    for src in (b, a):
        for dst, x in zip(static.args, whole(src)):
            dst.copy_(x)
        for name in ("perm_d", "inv_d", "gate_sa", "gate_swa"):
            getattr(static, name).copy_(getattr(src, name))
        graph.replay()
        src.check(out, path, 20, 30, what=path)
    assert sa.check_error(err) == sa.SA_OK


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("path", ["swa", "sa", "gated"])
def test_what_follows_a_call_finds_all_of_it_done(path, captured):
    """A call's kernels may run beside each other; whatever comes next in the
    stream may not: it reads whole results, and may overwrite the inputs."""
    new, total = [300, 1, 1, 700, 2, 1], [2100, 900, 1500, 1400, 33, 1]
    b = Batch(new, total, 8, 2, 128, 48, seed=12, perm_len=2200)
    out = torch.empty(b.t, 8, 128, dtype=torch.bfloat16, device="cuda")
    err = err_word()
    kept = [torch.empty_like(out) for _ in range(3)]
    inputs = [b.k, b.v, b.args[4]]
    saved = [x.clone() for x in inputs]
    spoiled = [torch.full_like(x, 7) for x in inputs]

    def step():
        for x in kept:
            for t, y in zip(inputs, saved):
                t.copy_(y)
            b.run(path, 300, 1000, out=out, err=err, max_new=700)
            for t, y in zip(inputs, spoiled):
                t.copy_(y)
            x.copy_(out)
            out.zero_()

    step()
    if captured:
        torch.cuda.synchronize()
        for x in kept:
            x.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graph.replay()
        graph.replay()
    for t, y in zip(inputs, saved):
        t.copy_(y)
    assert sa.check_error(err) == sa.SA_OK
    b.check(kept[0], path, 300, 1000, weight_bits=8, what=path)
    assert torch.equal(kept[0], kept[1]) and torch.equal(kept[0], kept[2])


@pytest.fixture(params=["short", "long"])
def way(request, monkeypatch):
    """Both ways from Python into the library."""
    from stochastic_sliding_window_gb300 import _paged
    _paged._get_native()
    assert _paged._native, "paged_call.cpp was not built"
    if request.param == "long":
        monkeypatch.setattr(_paged, "_native", False)
    return request.param


def test_both_ways_take_the_same_arguments(way, monkeypatch):
    from stochastic_sliding_window_gb300 import _paged
    shapes = dict(stride_q=64, pair_pages=True, behind=2)
    b = Batch([1, 3, 40], [700, 90, 41], 8, 2, 128, 16, seed=6, perm_len=800, **shapes)
    out = torch.zeros(b.t + 2, 8, 128, dtype=torch.bfloat16, device="cuda")
    err = err_word()
    for path in ("swa", "sa", "gated"):
        kw = dict(max_new=40, softmax_scale=0.25, err=err)
        got = b.run(path, 30, 50, **kw)
        assert b.run(path, 30, 50, out=out, **kw) is out
        assert got.shape == out.shape and got.dtype == torch.bfloat16 and not got.requires_grad
        b.check(got, path, 30, 50, weight_bits=8, scale=0.25, what=path)
        # (np.int64 is no int: the long way)
        assert torch.equal(b.run(path, np.int64(30), 50, **kw)[:b.t], got[:b.t])
        with monkeypatch.context() as m:
            m.setattr(_paged, "_native", False)
            assert torch.equal(b.run(path, 30, 50, **kw)[:b.t], got[:b.t])
    assert sa.check_error(err) == sa.SA_OK


def test_both_ways_plan_and_append(way):
    table, free = i32(np.full((2, 4), -1)), i32(np.arange(9))
    p = sa.paged_plan(i32([5, 1]), i32([0, 0]), table, free, i32([9]), page_size=4, num_pages=9, max_tokens=7)
    assert p._fields == ("q_start", "seq_lens", "slots", "positions", "counts")
    assert [x.tolist() for x in p] == [[0, 5, 6], [5, 1], [32, 33, 34, 35, 28, 24, -1], [0, 1, 2, 3, 4, 0, -1], [6, 3, 6]]
    assert all(x.is_contiguous() and x.dtype == torch.int32 for x in p)
    kv = bf16(np.random.default_rng(0).standard_normal((7, 2, 3, 64)))
    kc = torch.zeros(9, 4, 3, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    assert sa.paged_append(kv[:, 0], kv[:, 1], kc, vc, p.slots) is None
    rows = p.slots[:6].long()
    assert torch.equal(kc.view(-1, 3, 64)[rows], kv[:6, 0]) and torch.equal(vc.view(-1, 3, 64)[rows], kv[:6, 1])
    q = sa.paged_append(kv[:, 0], kv[:, 1], kc, vc, p.slots, p.positions, rope_base=100, q=kv[:, 1])
    assert q.shape == (7, 3, 64) and torch.equal(q[:1], kv[:1, 1])
    assert sa.paged_append(kv[:, 0], kv[:, 1], kc, vc, p.slots, p.positions, rope_base=100.0, q=kv[:, 1], q_out=q) is q


def test_both_ways_refuse(way):
    b = Batch([1, 3], [70, 9], 8, 2, 64, 16, seed=6, perm_len=80)
    q, k, v, table, start, lens = b.args
    run = lambda *a, **kw: sa.sa_paged_forward(*a, b.perm_d, b.inv_d, **{"window": 4, **kw})
    for bad, kind in [((q.float(), k, v, table, start, lens), TypeError), ((q, k, v.half(), table, start, lens), TypeError),
                      ((q, k, v[:, :8], table, start, lens), ValueError), ((q, k, v, table.long(), start, lens), TypeError),
                      ((q, k, v, table[:1], start, lens), ValueError), ((q, k, v, table, start[:2], lens), ValueError),
                      ((q, k, v, table.cpu(), start, lens), ValueError), ((q.cpu(), k, v, table, start, lens), ValueError),
                      ((q[:, :, :32], k, v, table, start, lens), ValueError), ((None, k, v, table, start, lens), TypeError)]:
        with pytest.raises(kind):
            run(*bad)
    for kw in (dict(window=0), dict(kernel=9), dict(kernel=sa.PAGED_TILES), dict(out=q)):
        with pytest.raises(RuntimeError):
            run(*b.args, **kw)
    with pytest.raises(ValueError):
        run(*b.args, out=torch.empty(3, 8, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        run(*b.args, err=torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError):
        sa.paged_plan(i32([1]), i32([0]), table, i32([0]), i32([1]), page_size=4, num_pages=1, max_tokens=1)
    with pytest.raises(ValueError):
        sa.paged_append(k[0, :1], v[0, :1], k, v, i32([0]), rope_base=10.0)


def test_given_streams():
    """A call on a stream of its own, ordered by the caller."""
    b = Batch([1, 1], [700, 90], 8, 2, 128, 16, seed=6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = b.run("swa", ALL, stream=side)
    raw = b.run("swa", ALL, stream=side.cuda_stream)
    side.synchronize()
    b.check(out, "swa", ALL)
    assert torch.equal(out, raw)


def test_no_tokens():
    b = Batch([1], [5], 4, 2, 64, 16)
    q = b.q[:0]
    out = sa.swa_paged_forward(q, *b.args[1:4], i32([0, 0]), i32([5]), window=4)
    assert out.shape == (0, 4, 64)
    sa.paged_append(b.k[0, :0], b.v[0, :0], b.k, b.v, i32(np.zeros(0)))
