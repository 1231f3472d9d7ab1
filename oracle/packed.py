"""Plain fp64 restatements of the rotation, of rows appended to a KV cache, and of the 4-bit cache's format (test
infrastructure; no code shared with the library).

A scale's byte has five exponent and three mantissa bits; a code is one of 16.  Both are found by search in the lists of all
their values.
"""
from __future__ import annotations

import numpy as np

BAD_LAYOUT, NONFINITE, SLOT_RANGE = 8, 2, 128
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MOST = 0xE2
SCALES = np.array([(b % 8) * 2.0 ** -17 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 18) for b in range(MOST + 1)])
LARGEST = 6.0 * SCALES[MOST]


def _nearest(a, grid):
    """Indices of the nearest entries of a rising grid; half way, the even index."""
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    up, down = grid[hi] - a, a - grid[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantize(x):
    """x [..., dim]: codes [..., dim] (0..15), scale bytes [..., dim / 16], and their values."""
    x = np.asarray(x, np.float64)
    y = x.reshape(*x.shape[:-1], -1, 16)
    y = np.clip(np.where(np.isnan(y), 0.0, y), -LARGEST, LARGEST)
    byte = _nearest(np.abs(y).max(-1), 6.0 * SCALES)
    s = SCALES[byte][..., None]
    borders = (MAGNITUDES[1:] + MAGNITUDES[:-1]) / 2
    a = np.abs(y)
    code = np.zeros(y.shape, np.uint8)
    for i in range(7):
        code += ((a > borders[i] * s) | ((a == borders[i] * s) & (i % 2 == 1))) & (s > 0)
    value = np.where(y < 0, -1.0, 1.0) * MAGNITUDES[code] * s
    return (code | ((y < 0) << 3).astype(np.uint8)).reshape(x.shape), byte.astype(np.uint8), value.reshape(x.shape)


def block_bytes(page, dim):
    return -(-page * dim * 9 // 128) * 16


def blocks(k_codes, k_scales, v_codes, v_scales):
    """Codes [layers, pages, page, heads, dim] and scales [.., dim / 16] as blocks [layers, pages, heads, bytes]."""
    L, P, S, H, D = k_codes.shape
    out = np.zeros((L, P, H, block_bytes(S, D)), np.uint8)
    at = 0
    for c in (k_codes, v_codes):
        b = (c[..., 0::2] | (c[..., 1::2] << 4)).transpose(0, 1, 3, 2, 4).reshape(L, P, H, -1)
        out[..., at:at + b.shape[-1]] = b
        at += b.shape[-1]
    for s in (k_scales, v_scales):
        b = s.transpose(0, 1, 3, 2, 4).reshape(L, P, H, -1)
        out[..., at:at + b.shape[-1]] = b
        at += b.shape[-1]
    return out


def unblock(data, page, dim):
    """The reverse: k_codes, k_scales, v_codes, v_scales as in blocks()."""
    L, P, H, _ = data.shape
    out, at = [], 0
    for _ in range(2):
        b = data[..., at:at + page * dim // 2].reshape(L, P, H, page, dim // 2).transpose(0, 1, 3, 2, 4)
        out.append(np.stack([b & 15, b >> 4], -1).reshape(L, P, page, H, dim))
        at += page * dim // 2
    for _ in range(2):
        out.append(data[..., at:at + page * dim // 16].reshape(L, P, H, page, dim // 16).transpose(0, 1, 3, 2, 4))
        at += page * dim // 16
    return tuple(np.ascontiguousarray(out[i]) for i in (0, 2, 1, 3))


def values(codes, scales):
    s = SCALES[np.minimum(scales, MOST)].repeat(16, -1)
    return np.where(codes >= 8, -1.0, 1.0) * MAGNITUDES[codes & 7] * s


def _two_pi(bits):
    """2 pi times 2^bits, from Machin's 16 arctan(1/5) - 4 arctan(1/239) in whole numbers."""
    def arctan_of_one_over(n):
        one = 1 << (bits + 20)
        term, total, i = one // n, 0, 1
        while term:
            total += term // i if i % 4 == 1 else -(term // i)
            term //= n * n
            i += 2
        return total
    return (32 * arctan_of_one_over(5) - 8 * arctan_of_one_over(239)) >> 20


def angles(positions, inv_freq):
    """position * inv_freq [rows, pairs], where fp64 does not hold that exactly less whole turns, by whole numbers."""
    pos, f = np.asarray(positions, np.int64), np.asarray(inv_freq, np.float64)
    out = pos[:, None].astype(np.float64) * f
    for r in np.nonzero(np.abs(pos.astype(np.float64)) >= 2.0 ** 29)[0]:  # (a float has 24 bits)
        for i, x in enumerate(f):
            a, b = float(x).as_integer_ratio()
            n = (int(pos[r]) * a << 256) // b
            n -= (2 * n + _TURN) // (2 * _TURN) * _TURN  # less the nearest number of turns
            out[r, i] = float(n) / 2.0 ** 256
    return out


_TURN = _two_pi(256)


def rotate(x, positions, inv_freq, interleaved=False, magnitude=1.0):
    """x [rows, heads, dim]: pairs of columns as complex numbers, turned; and |x| + |y| of each column's pair (0: left alone)."""
    x = np.asarray(x, np.float64)
    n = len(inv_freq)
    angle = angles(positions, inv_freq)[:, None]
    turn = magnitude * (np.cos(angle) + 1j * np.sin(angle))
    out, mag = x.copy(), np.zeros_like(x)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    with np.errstate(invalid="ignore"):
        z = (x[..., a] + 1j * x[..., b]) * turn
    out[..., a], out[..., b] = z.real, z.imag
    mag[..., a] = mag[..., b] = abs(magnitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, mag


def places(table, seq_lens, rows_of, page, pages, total, row_slots=None, max_len=None):
    """Slot (-1: outside the cache, -2: a row of no request) and number of each row, and the requests' status.

    rows_of: (first row, one past the last) of each request."""
    slot, number, status = np.full(total, -2, np.int64), np.zeros(total, np.int64), np.zeros(len(rows_of), np.uint32)
    for b, (lo, hi) in enumerate(rows_of):
        L = 0 if seq_lens is None else int(seq_lens[b])
        if lo < 0 or hi < lo or hi > total or (max_len is not None and hi - lo > max_len):
            status[b] |= BAD_LAYOUT
            continue
        if L < 0:
            status[b] |= BAD_LAYOUT
            continue
        for r in range(lo, hi):
            number[r] = r - lo
            if row_slots is not None:
                s = int(row_slots[r])
                slot[r] = s if 0 <= s < pages * page else -1
            else:
                x = L + r - lo
                p = int(table[b][x // page]) if x // page < table.shape[1] else -1
                slot[r] = p * page + x % page if 0 <= p < pages else -1
            if slot[r] == -1:
                status[b] |= SLOT_RANGE
    return slot, number, status
