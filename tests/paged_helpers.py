"""Inputs and tolerances of the paged-cache tests."""

from __future__ import annotations

import numpy as np
import torch

import oracle
import stochastic_sliding_window_gb300 as sa


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(torch.bfloat16)


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Batch:
    """A ragged batch over a cache whose pages are shuffled; every cache row
    that no position names holds NaN, and so do the rows of q and out behind
    the last request."""

    def __init__(self, new, total, hq, hkv, d, page, seed=0, behind=0, stride_q=0, pair_pages=False,
                 perm_len=0, shared_perm=False, spread=1.0):
        rng = np.random.default_rng(seed)
        self.new, self.total, b = new, total, len(new)
        self.hq, self.hkv, self.d, self.page = hq, hkv, d, page
        need = [-(-t // page) for t in total]
        width = max(need) + 1
        self.num_pages = sum(need) + 3
        ids = rng.permutation(self.num_pages)
        self.table = np.full((b, width), -1, dtype=np.int64)
        at = 0
        for r in range(b):
            self.table[r, :need[r]] = ids[at:at + need[r]]
            at += need[r]
        nan = torch.full((self.num_pages, 2, page, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        kc = np.full((self.num_pages, page, hkv, d), np.nan, dtype=np.float32)
        vc = kc.copy()
        for r in range(b):
            j = np.arange(total[r])
            kc[self.table[r, j // page], j % page] = rng.standard_normal((total[r], hkv, d))
            vc[self.table[r, j // page], j % page] = rng.standard_normal((total[r], hkv, d))
        if pair_pages:  # one array of pages, each K then V
            nan[:, 0], nan[:, 1] = bf16(kc), bf16(vc)
            self.k, self.v = nan[:, 0], nan[:, 1]
        else:
            self.k, self.v = bf16(kc), bf16(vc)
        t = sum(new)
        self.t = t
        wide = torch.full((t + behind, hq * d + stride_q), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:t, :hq * d] = bf16(rng.standard_normal((t, hq * d)) * spread)
        self.q = wide[:, :hq * d].unflatten(1, (hq, d)) if stride_q else wide.view(-1, hq, d)
        self.q_start = np.concatenate([[0], np.cumsum(new)])
        self.args = (self.q, self.k, self.v, i32(self.table), i32(self.q_start), i32(total))
        if perm_len:
            rows = 1 if shared_perm else b
            self.perm = np.stack([oracle.make_perm(seed, 1, r, perm_len) for r in range(rows)])
            self.perm_d = i32(self.perm)
            self.inv_d = sa.sa_inverse_perm(self.perm_d)
        self.gate_sa = torch.from_numpy(rng.standard_normal((t + behind, hq)).astype(np.float32)).cuda()
        self.gate_swa = torch.from_numpy(rng.standard_normal((t + behind, hq)).astype(np.float32)).cuda()

    def run(self, path, window, window_swa=0, **kw):
        if path == "swa":
            return sa.swa_paged_forward(*self.args, window=window, **kw)
        if path == "sa":
            return sa.sa_paged_forward(*self.args, self.perm_d, self.inv_d, window=window, **kw)
        return sa.sa_swa_gated_paged_forward(*self.args, self.perm_d, self.inv_d, self.gate_sa,
                                             self.gate_swa, window=window, window_swa=window_swa, **kw)

    def want(self, path, window, window_swa=0, **kw):
        f = lambda x: x.float().cpu().numpy()
        return oracle.paged_attention(path, f(self.q[:self.t]), f(self.k), f(self.v), self.table,
                                      self.q_start, self.total, window, window_swa,
                                      getattr(self, "perm", None), f(self.gate_sa)[:self.t],
                                      f(self.gate_swa)[:self.t], **kw)

    def check(self, got, path, window, window_swa=0, weight_bits=16, what="", **kw):
        """Every element within the rounding errors of the computation.

        With e the fp32 half step 2^-24: a score is a sum of d products held
        in fp32, off by at most d e times the sum of their sizes, at most
        scale |q| |k|; scaling by log2(e), the subtraction of the maximum and
        2^x (whose result is good to 2^-22) add a few e of the score's size.
        That relative error ds of each weight enters the result twice (weight
        and sum), as does the rounding of the weights (half a step of
        2^-weight_bits; twice since the sum is of the unrounded ones).  The
        products' sums run over at most L terms in fp32.  All of these
        multiply sum |weight value|; the result is rounded once, by half a
        step of bf16, 2^-8 of itself.
        """
        want, spread = self.want(path, window, window_swa, **kw)
        f = lambda x: x.float().cpu().numpy().astype(np.float64)
        scale = kw.get("scale") or self.d ** -0.5
        qn = np.linalg.norm(f(self.q[:self.t]), axis=-1).max()
        kn = np.nanmax(np.linalg.norm(f(self.k), axis=-1))
        e = 2.0 ** -24
        ds = (self.d + 8) * e * scale * qn * kn * 1.4427 + 2.0 ** -21
        rel = 2 * ds + 2.0 ** -weight_bits + (max(self.total) + 8) * e
        bar = rel * spread + 2.0 ** -8 * (np.abs(want) + rel * spread) + 1e-30
        g = f(got)
        assert g.shape[0] >= self.t
        off = np.abs(g[:self.t] - want)
        assert np.isfinite(g[:self.t]).all(), f"{what}: non-finite rows"
        worst = float((off / bar).max()) if off.size else 0.0
        assert worst <= 1.0, f"{what}: error {worst:.2f} times the bound"
        return worst
