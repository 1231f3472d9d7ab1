"""Inputs shared by the tests of the calls that fill and read a KV cache, and of the 4-bit cache."""
from __future__ import annotations

import numpy as np
import torch

from oracle import packed
from tests.serving_cases import BF16, F32, AttentionCase


class PackedAttentionCase(AttentionCase):
    """An AttentionCase whose cache is held in 4 bits; every entry that no request owns has bytes of ones."""

    def __init__(self, *args, gain=1.0, **kw):
        super().__init__(*args, F32, **kw)
        free = torch.isnan(self.k[:, :, :, :1, :1]).numpy()
        self.q, self.dtype = self.q.to(BF16), BF16
        held = []
        for name in ("k", "v"):
            x = gain * torch.nan_to_num(getattr(self, name)).double().numpy()
            codes, scales, value = packed.quantize(x)
            codes[np.broadcast_to(free, codes.shape)] = 15
            scales[np.broadcast_to(free, scales.shape)] = 255
            value[np.broadcast_to(free, value.shape)] = np.nan
            held += [codes, scales]
            setattr(self, name, torch.from_numpy(value))
        self.blocks = packed.blocks(*held)

    def cache(self, sv, device="cuda"):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)
        data = dev(self.blocks)
        if self.head_major:  # heads before pages in memory
            data = data.transpose(1, 2).contiguous().transpose(1, 2)
        self.data, self.dtable = data, dev(self.table)
        return sv.PackedKvCache(data, self.dtable, page_size=self.page, head_dim=self.q.shape[2])

    def oracle(self):
        """With what weights in half floats may add to a correct computation's error: a weight's own 2^-12 is below the 2^-8 that
        the bounds count for it, but a small one is a whole number of steps of 2^-24, half of one off, where the largest weight of
        the row is 2^6 at least (a reference is set that far below a maximum).  So each of the keys seen may add 2^-31 of its |v|."""
        o = super().oracle()
        most = np.nan_to_num(self.v[self.layer].abs().numpy()).max()
        o["mag"] = o["mag"] + 2.0 ** -31 * o["count"][:, None, None] * most / 2.0 ** -8
        return o

    def run(self, sv, out=None, ws=None, stream=None, scale=None):
        dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
        return sv.paged_attention(self.q.cuda(), self.cache(sv), dev(np.asarray(self.lens, np.int64)), layer=self.layer,
                                  max_len=self.max_len, cu_seqlens=dev(self.cu), row_slots=dev(self.row_slots),
                                  mask=dev(self.mask), scale=self.scale if scale is None else scale, out=out, ws=ws,
                                  stream=stream)


# A rotated value's error in fp32: sine and cosine by 2^-23 (two units in the last place of a value of at most 1, with the
# magnitude's rounding another 2^-24), a product and a multiply-add by 2^-24 each.
ROTATED = 3 * 2.0 ** -23


class AppendCase:
    """Rows appended to a cache with random contents, in random page order."""

    def __init__(self, lens, rows, heads, kv_heads, dim, page, dtype, *, is_packed=False, ragged=False, staged=False,
                 positions=None, pairs=None, interleaved=False, magnitude=1.0, spare_rows=0, layers=1, layer=0, seed=0,
                 rotation=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        rows = [rows] * B if isinstance(rows, int) else list(rows)
        self.lens, self.rows, self.max_len = list(lens), rows, max(max(rows), 1)
        R = sum(rows) + spare_rows
        room = [max(1, -(-(L + (0 if staged else r)) // page)) for L, r in zip(lens, rows)]
        spare = -(-R // page) if staged else 0
        self.pages = sum(room) + spare + 2
        order = rng.permutation(self.pages)
        self.table = np.full((B, max(room)), -7, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :room[b]] = order[at:at + room[b]]
            at += room[b]
        self.row_slots = None
        if staged:
            self.row_slots = np.concatenate([order[at + i] * page + np.arange(page) for i in range(spare)])[:R].astype(np.int64)
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32) if ragged else None
        self.heads, self.kv_heads, self.dim, self.page, self.dtype, self.is_packed = heads, kv_heads, dim, page, dtype, is_packed
        self.layers, self.layer, self.total, self.interleaved, self.magnitude = layers, layer, R, interleaved, magnitude
        self.qkv = torch.randn(R, heads + 2 * kv_heads, dim, generator=g).to(dtype)
        self.positions = None if positions is None else np.asarray(positions, np.int64)
        n = dim // 2 if pairs is None else pairs
        self.inv_freq = (10000.0 ** (-np.arange(n) / max(n, 1))).astype(np.float32) if rotation else None
        if is_packed:
            self.before = rng.integers(0, 256, (layers, self.pages, kv_heads, packed.block_bytes(page, dim)), dtype=np.uint8)
        else:
            self.before = [torch.randn(layers, self.pages, page, kv_heads, dim, generator=g).to(dtype) for _ in range(2)]

    def make(self, sv):
        dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
        d = {"table": dev(self.table), "seq_lens": dev(np.asarray(self.lens, np.int64)), "cu": dev(self.cu),
             "slots": dev(self.row_slots), "positions": dev(self.positions), "qkv": self.qkv.cuda()}
        if self.is_packed:
            d["data"] = dev(self.before)
            d["cache"] = sv.PackedKvCache(d["data"], d["table"], page_size=self.page, head_dim=self.dim, dtype=self.dtype)
        else:
            d["k"], d["v"] = (t.cuda() for t in self.before)
            d["cache"] = sv.PagedKvCache(d["k"], d["v"], d["table"])
        d["rotation"] = None if self.inv_freq is None else sv.Rotation(dev(self.inv_freq), interleaved=self.interleaved,
                                                                       magnitude=self.magnitude)
        return d

    def append(self, sv, d, q=True, out=None, stream=None):
        H, G = self.heads, self.kv_heads
        x = d["qkv"]
        return sv.kv_append(d["cache"], x[:, H:H + G], x[:, H + G:], layer=self.layer, seq_lens=d["seq_lens"],
                            max_len=self.max_len, cu_seqlens=d["cu"], row_slots=d["slots"], positions=d["positions"],
                            rotation=d["rotation"], q=x[:, :H] if q else None, out=out, stream=stream)

    def read(self, sv, d, layer=0, out=None):
        return sv.kv_read(d["cache"], layer=layer, seq_lens=d["seq_lens"], max_len=self.max_len, cu_seqlens=d["cu"],
                          row_slots=d["slots"], rows=self.total, out=out)

    def oracle(self):
        H, G = self.heads, self.kv_heads
        x = self.qkv.double().numpy()
        if self.cu is None:
            spans = [(b * self.max_len, (b + 1) * self.max_len) for b in range(len(self.lens))]
        else:
            spans = [(int(self.cu[b]), int(self.cu[b + 1])) for b in range(len(self.lens))]
        slot, number, status = packed.places(self.table, self.lens, spans, self.page, self.pages, self.total, self.row_slots,
                                             self.max_len)
        pos = self.positions
        if pos is None:
            pos = np.zeros(self.total, np.int64)
            for b, (lo, hi) in enumerate(spans):
                if 0 <= lo <= hi <= self.total:
                    pos[lo:hi] = self.lens[b] + number[lo:hi]
        q, k, qm, km = x[:, :H], x[:, H:H + G], np.zeros_like(x[:, :H]), np.zeros_like(x[:, H:H + G])
        if self.inv_freq is not None:
            q, qm = packed.rotate(q, pos, self.inv_freq, self.interleaved, self.magnitude)
            k, km = packed.rotate(k, pos, self.inv_freq, self.interleaved, self.magnitude)
            if self.magnitude == 1.0:  # an angle of 0 changes nothing
                qm[pos == 0], km[pos == 0] = 0.0, 0.0
        if self.is_packed:
            odd = ~np.isfinite(x[:, H:]).all(axis=(1, 2))
            for b, (lo, hi) in enumerate(spans):
                for r in range(max(lo, 0), min(hi, self.total)):
                    if slot[r] >= 0 and odd[r]:
                        status[b] |= packed.NONFINITE
        return {"slot": slot, "status": status, "q": q, "q_err": ROTATED * qm, "k": k, "k_err": ROTATED * km,
                "v": x[:, H + G:]}


def near_border(x, err):
    """Whether a value within err of x may have another scale or code than x."""
    y, e = x.reshape(*x.shape[:-1], -1, 16), err.reshape(*err.shape[:-1], -1, 16)
    a = np.abs(y)
    top = a.max(-1)
    slack = e.max(-1)
    lo, hi = (packed._nearest(np.clip(t, 0, packed.LARGEST), 6.0 * packed.SCALES) for t in (top - slack, top + slack))
    s = packed.SCALES[lo][..., None]
    borders = (packed.MAGNITUDES[1:] + packed.MAGNITUDES[:-1]) / 2
    close = (np.abs(a[..., None] - borders * s[..., None]) <= e[..., None]).any(-1) & (e > 0)
    return (close | (lo != hi)[..., None]).reshape(x.shape)


def check_append(case, d, got, q=True):
    """The rotated queries, the stored rows, and that nothing else changed."""
    o = case.oracle()
    eps = 2.0 ** -8 if case.dtype == BF16 else 2.0 ** -24
    mine = o["slot"] > -2
    if q:
        out = got.q.double().cpu().numpy()
        assert (np.abs(out - o["q"]) <= eps * np.abs(o["q"]) + o["q_err"] + 1e-38)[mine].all()
    assert np.array_equal(got.dev_status.cpu().numpy().view(np.uint32), o["status"])
    rows = np.nonzero(o["slot"] >= 0)[0]
    at = o["slot"][rows]
    if not case.is_packed:
        for name, i, err in (("k", 0, o["k_err"][rows]), ("v", 1, None)):
            new = d[name].cpu()
            want = case.before[i].clone()
            flat = lambda t: t[case.layer].reshape(-1, case.kv_heads, case.dim)
            have = flat(new)[at].double().numpy()
            exact = o[name][rows]
            if err is None:
                assert np.array_equal(have, exact)
            else:
                assert (np.abs(have - exact) <= eps * np.abs(exact) + err + 1e-38).all()
            flat(want)[at] = flat(new)[at]
            assert torch.equal(new, want)
        return
    after = d["data"].cpu().numpy()
    parts, old = packed.unblock(after, case.page, case.dim), packed.unblock(case.before, case.page, case.dim)
    flat = lambda t: t[case.layer].reshape(case.pages * case.page, *t.shape[3:])
    for i, name in ((0, "k"), (2, "v")):
        codes, scales = flat(parts[i])[at], flat(parts[i + 1])[at]
        _, _, want = packed.quantize(o[name][rows])
        have = packed.values(codes, scales)
        err = o["k_err"][rows] if name == "k" else np.zeros_like(want)
        near = near_border(o[name][rows], err)
        assert np.array_equal(have[~near], want[~near])
        # (the oracle's numbers alone: a border is 1 part in 2^20 of its surroundings, but bf16 values that are turned by next to
        # nothing, at the first positions, lie on one themselves every 20th time or so)
        assert near.mean() < 0.1
        # near a border: the value of the neighbour, a step of the larger scale away at most
        step = packed.SCALES[np.maximum(scales, 1)].repeat(16, -1) * 2.25
        assert (np.abs(have - want) <= step)[near].all()
    for a, b in zip(parts, old):
        a, b = a.copy(), b.copy()
        flat(a)[at] = flat(b)[at] = 0
        assert np.array_equal(a, b)
