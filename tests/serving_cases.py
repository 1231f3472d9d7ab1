"""Inputs shared by the tests of the serving-side operators."""
from __future__ import annotations

import numpy as np
import torch

BF16, F32 = torch.bfloat16, torch.float32


def random_tree(rng, n):
    """Parents of a random tree whose nodes follow their parents, and its ancestor-or-self mask."""
    par = [-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, n)]
    mask = np.zeros((n, n), np.uint8)
    for i in range(n):
        j = i
        while j != -1:
            mask[i, j] = 1
            j = par[j]
    return par, mask


class AttentionCase:
    """A paged cache in random page order, every entry that no request owns poisoned with NaN."""

    def __init__(self, lens, rows, heads, kv_heads, dim, page, dtype, *, ragged=False, tree=False, staged=False,
                 head_major=False, layers=1, layer=0, seed=0, q_gain=2.0, poison=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        rows = [rows] * B if isinstance(rows, int) else list(rows)
        self.max_len, self.lens, self.rows = max(rows), list(lens), rows
        self.row0 = np.concatenate([[0], np.cumsum(rows)[:-1]]).tolist()
        R = sum(rows)
        room = [max(1, -(-(L + (0 if staged else r)) // page)) for L, r in zip(lens, rows)]
        spare = -(-R // page) if staged else 0
        pages = sum(room) + spare + 2
        order = rng.permutation(pages)
        self.table = np.full((B, max(room)), -7, np.int32)  # entries past a request's pages are never valid pages
        at, owned = 0, np.zeros(pages * page, bool)
        for b in range(B):
            self.table[b, :room[b]] = order[at:at + room[b]]
            at += room[b]
            for x in range(lens[b] + (0 if staged else rows[b])):
                owned[self.table[b, x // page] * page + x % page] = True
        self.row_slots = None
        if staged:
            self.row_slots = np.concatenate([order[at + i] * page + np.arange(page) for i in range(spare)])[:R].astype(np.int64)
            owned[self.row_slots] = True
        shape = (layers, pages, page, kv_heads, dim)
        k = torch.randn(shape, generator=g).to(dtype)
        v = torch.randn(shape, generator=g).to(dtype)
        if poison:
            free = torch.from_numpy(~owned).view(pages, page)
            k[:, free] = float("nan")
            v[:, free] = float("nan")
        self.mask = None
        if tree:
            self.mask = np.zeros((B, self.max_len, self.max_len), np.uint8)
            for b in range(B):
                self.mask[b, :rows[b], :rows[b]] = random_tree(rng, rows[b])[1]
        self.q = (q_gain * torch.randn(R, heads, dim, generator=g)).to(dtype)
        self.k, self.v, self.layer, self.scale = k, v, layer, dim ** -0.5
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32) if ragged else None
        self.head_major, self.page, self.dtype = head_major, page, dtype

    def run(self, sv, out=None, ws=None, stream=None, scale=None):
        def layout(t):  # head-major pages: the same axes over another order in memory
            t = t.cuda()
            return t.transpose(2, 3).contiguous().transpose(2, 3) if self.head_major else t
        dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.dk, self.dv, self.dtable = layout(self.k), layout(self.v), dev(self.table)
        cache = sv.PagedKvCache(self.dk, self.dv, self.dtable)
        return sv.paged_attention(self.q.cuda(), cache, dev(np.asarray(self.lens, np.int64)), layer=self.layer,
                                  max_len=self.max_len, cu_seqlens=dev(self.cu), row_slots=dev(self.row_slots),
                                  mask=dev(self.mask), scale=self.scale if scale is None else scale, out=out, ws=ws,
                                  stream=stream)

    def oracle(self):
        from oracle import serving
        f = lambda t: t.double().numpy()
        return serving.attention(f(self.q), f(self.k[self.layer]), f(self.v[self.layer]), self.table, self.lens,
                                 self.row0, self.rows, self.scale, self.row_slots, self.mask)


def attention_bounds(o, dim, dtype):
    """Bounds of |out - exact| and |lse - exact| of a correct fp32 computation (bf16: with weights and result rounded).

    A score is a sum of dim products (relative to its largest sum of magnitudes), an exponential costs 2^-21, the sums
    over n keys n 2^-24; a weight's relative error moves the result by that share of sum p |v|, twice with the
    normaliser's.  bf16 rounds each weight and the result by at most 2^-8 of themselves."""
    n = o["count"][:, None].astype(np.float64)
    score = (dim + 8) * 2.0 ** -24 * o["smax"] + 2.0 ** -21
    sums = (n + 16) * 2.0 ** -24
    rel = 2 * score + 2 * sums
    tol = rel[..., None] * o["mag"]
    if dtype == BF16:
        tol = tol + 2.0 ** -8 * o["mag"] + 2.0 ** -8 * np.abs(o["out"])
    with np.errstate(invalid="ignore"):
        lse = score + sums + 2.0 ** -22 * np.where(np.isfinite(o["lse"]), np.abs(o["lse"]), 0.0) + 2.0 ** -22
    return tol + 1e-30, lse


def check_attention(case, got):
    o = case.oracle()
    tol, lse_tol = attention_bounds(o, case.q.shape[2], case.dtype)
    out, lse = got.out.double().cpu().numpy(), got.lse.double().cpu().numpy()
    assert np.array_equal(np.isnan(out), np.isnan(o["out"]))
    assert np.array_equal(np.isneginf(lse), np.isneginf(o["lse"]))
    fine = np.isfinite(o["out"])
    assert (np.abs(out - o["out"])[fine] <= tol[fine]).all(), float((np.abs(out - o["out"]) / tol)[fine].max())
    fine = np.isfinite(o["lse"])
    assert (np.abs(lse[fine] - o["lse"][fine]) <= lse_tol[fine]).all()
    assert np.array_equal(got.dev_status.cpu().numpy().view(np.uint32), o["status"])
