"""Refusals of the calls that fill and read a KV cache and of the 4-bit cache's (no GPU): the binding's argument checks, run on CPU
tensors with the library's entry points replaced by stubs, and the library's own, which come before anything is enqueued.  And
the oracle of the 4-bit format against direct formulas."""
import ctypes
import os
import sys

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from oracle import packed  # noqa: E402
from reject_row_vocab_gb300 import specverify as sv  # noqa: E402

ENTRY = ("spec_verify_kv_append", "spec_verify_packed_kv_append", "spec_verify_kv_read", "spec_verify_packed_kv_read",
         "spec_verify_packed_attention", "spec_verify_packed_kv_commit", "spec_verify_paged_attention", "spec_verify_kv_commit")
BF16, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


class _StubLib:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name in ENTRY:
            return lambda *a: self.calls.append((name, a)) or 0
        return getattr(self.real, name)


@pytest.fixture(scope="module")
def lib():
    from reject_row_vocab_gb300 import _build
    _build.build()
    return sv.load_library()


@pytest.fixture
def stub(lib, monkeypatch):
    s = _StubLib(lib)
    monkeypatch.setattr(sv, "load_library", lambda: s)
    monkeypatch.setattr(sv, "_call_stream", lambda s, d: None)
    monkeypatch.setattr(sv, "_require_cache", lambda c: None)
    return s


def _table(batch=3, pages=4):
    return torch.zeros(batch, pages, dtype=I32)


def _whole(layers=2, pages=6, page=4, heads=2, dim=32, dtype=BF16):
    t = lambda: torch.zeros(layers, pages, page, heads, dim, dtype=dtype)
    return sv.PagedKvCache(t(), t(), _table())


def _packed(layers=2, pages=6, page=4, heads=2, dim=32, dtype=BF16):
    return sv.PackedKvCache.allocate(layers, pages, heads, page, dim, _table(), dtype)


CACHES = pytest.mark.parametrize("make", [_whole, _packed])


def _append(cache, **kw):
    a = dict(k=torch.zeros(6, 2, 32, dtype=BF16), v=torch.zeros(6, 2, 32, dtype=BF16), seq_lens=torch.zeros(3, dtype=I64),
             q=torch.zeros(6, 4, 32, dtype=BF16), rotation=sv.Rotation(torch.ones(16)),
             out=sv.KvAppendOutputs.allocate(6, 4, 32, 3, device="cpu"))
    a.update(kw)
    return sv.kv_append(cache, a.pop("k"), a.pop("v"), **a)


@CACHES
@pytest.mark.parametrize("good", [
    dict(), dict(max_len=2), dict(max_len=1), dict(q=None, out=None), dict(rotation=None), dict(layer=1),
    dict(row_slots=torch.zeros(6, dtype=I64)), dict(cu_seqlens=torch.zeros(4, dtype=I32), max_len=5),
    dict(seq_lens=None, row_slots=torch.zeros(6, dtype=I64), positions=torch.zeros(6, dtype=I64),
         out=sv.KvAppendOutputs.allocate(6, 4, 32, 6, device="cpu")),
    dict(k=torch.zeros(6, 4, 64, dtype=BF16)[:, ::2, :32]), dict(rotation=sv.Rotation(torch.zeros(0))),
    dict(out=None)])
def test_append_passes_what_it_takes(stub, make, good):
    out = _append(make(), **good)
    name, args = stub.calls[0]
    assert name == ("spec_verify_packed_kv_append" if make is _packed else "spec_verify_kv_append")
    assert args[0] is not None and out.dev_status.numel() >= 3


@CACHES
@pytest.mark.parametrize("bad,exc", [
    (dict(k=torch.zeros(6, 64, dtype=BF16)), ValueError), (dict(k=torch.zeros(6, 2, 32)), TypeError),
    (dict(k=torch.zeros(6, 3, 32, dtype=BF16)), ValueError), (dict(v=torch.zeros(5, 2, 32, dtype=BF16)), ValueError),
    (dict(v=torch.zeros(6, 2, 64, dtype=BF16)[:, :, ::2]), ValueError), (dict(v=None), ValueError),
    (dict(q=torch.zeros(5, 4, 32, dtype=BF16)), ValueError), (dict(q=torch.zeros(6, 4, 64, dtype=BF16)), ValueError),
    (dict(q=torch.zeros(6, 4, 32)), TypeError), (dict(q=7), ValueError),
    (dict(seq_lens=torch.zeros(3, dtype=I32)), TypeError), (dict(seq_lens=torch.zeros(4, dtype=I64)), ValueError),
    (dict(seq_lens=None), ValueError), (dict(seq_lens=None, row_slots=torch.zeros(6, dtype=I64)), ValueError),
    (dict(max_len=3), ValueError), (dict(cu_seqlens=torch.zeros(4, dtype=I32)), ValueError),
    (dict(cu_seqlens=torch.zeros(4, dtype=I64), max_len=2), TypeError),
    (dict(cu_seqlens=torch.zeros(5, dtype=I32), max_len=2), ValueError),
    (dict(row_slots=torch.zeros(5, dtype=I64)), ValueError), (dict(positions=torch.zeros(5, dtype=I64)), ValueError),
    (dict(positions=torch.zeros(6, dtype=I32)), TypeError), (dict(rotation=torch.ones(16)), TypeError),
    (dict(out=sv.KvAppendOutputs(q=None, dev_status=torch.zeros(3, dtype=I32))), ValueError),
    (dict(out=sv.KvAppendOutputs.allocate(6, 3, 32, 3, device="cpu")), ValueError),
    (dict(out=sv.KvAppendOutputs.allocate(6, 4, 32, 2, device="cpu")), ValueError)])
def test_append_refuses(stub, make, bad, exc):
    with pytest.raises(exc):
        _append(make(), **bad)
    assert not stub.calls


@CACHES
def test_more_requests_than_the_page_table_has(stub, make):
    with pytest.raises(ValueError):
        _append(make(), k=torch.zeros(8, 2, 32, dtype=BF16), v=torch.zeros(8, 2, 32, dtype=BF16), q=None,
                seq_lens=torch.zeros(4, dtype=I64), out=None)
    _append(make(), k=torch.zeros(8, 2, 32, dtype=BF16), v=torch.zeros(8, 2, 32, dtype=BF16), q=None,  # places given as slots
            seq_lens=torch.zeros(4, dtype=I64), row_slots=torch.zeros(8, dtype=I64), out=None)


@CACHES
def test_read(stub, make):
    cache, lens = make(), torch.zeros(3, dtype=I64)
    r = sv.kv_read(cache, layer=1, seq_lens=lens, max_len=2)
    assert r.k.shape == (6, 2, 32) and r.k.dtype == BF16
    assert sv.kv_read(cache, seq_lens=lens, max_len=2).v.shape == (2, 6, 2, 32)
    assert sv.kv_read(cache, layer=0, seq_lens=lens, cu_seqlens=torch.zeros(4, dtype=I32), max_len=9, rows=11).k.shape[0] == 11
    assert sv.kv_read(cache, layer=0, row_slots=torch.zeros(5, dtype=I64)).k.shape[0] == 5
    n = len(stub.calls)
    out = sv.KvReadOutputs.allocate(6, 2, 32, 3, device="cpu")
    for bad, exc in ((dict(seq_lens=lens), ValueError), (dict(seq_lens=lens, cu_seqlens=torch.zeros(4, dtype=I32), max_len=2), ValueError),
                     (dict(max_len=2), ValueError), (dict(seq_lens=lens, max_len=3, out=out, layer=0), ValueError),
                     (dict(seq_lens=lens, out=out), ValueError),
                     (dict(seq_lens=lens, layer=0, out=sv.KvReadOutputs.allocate(6, 2, 32, 3, F32, device="cpu")), TypeError),
                     (dict(seq_lens=lens, layer=0, out=sv.KvReadOutputs(k=out.k, v=torch.zeros(6, 2, 64, dtype=BF16)[:, :, :32],
                                                                       dev_status=out.dev_status)), ValueError)):
        with pytest.raises(exc):
            sv.kv_read(cache, **bad)
    assert len(stub.calls) == n


def test_packed_cache_refuses():
    t = _table()
    data = torch.zeros(1, 2, 2, 144, dtype=torch.uint8)
    sv.PackedKvCache(data, t, page_size=4, head_dim=32)
    for args, kw, exc in (((data.int(), t), {}, TypeError), ((data[0], t), {}, ValueError), ((data, t[0]), {}, ValueError),
                          ((data, t.long()), {}, TypeError), ((data, t), dict(dtype=torch.float16), TypeError),
                          ((data, t), dict(page_size=5), ValueError), ((data, t), dict(head_dim=48), ValueError),
                          ((data, t), dict(head_dim=288), ValueError), ((data, t), dict(page_size=0), ValueError),
                          ((data[..., ::2], t), dict(page_size=2), ValueError)):
        with pytest.raises(exc):
            sv.PackedKvCache(*args, **{**dict(page_size=4, head_dim=32), **kw})


def test_rotation_refuses():
    for bad, exc in ((torch.ones(2, 2), ValueError), (torch.ones(2, dtype=torch.float64), TypeError), ([1.0], ValueError),
                     (torch.ones(4)[::2], ValueError)):
        with pytest.raises(exc):
            sv.Rotation(bad)


def test_calls_need_a_gpu():
    with pytest.raises(ValueError, match="CUDA"):
        _append(_packed())
    with pytest.raises(TypeError):
        _append(torch.zeros(3))


def test_attention_and_commit_take_either_cache(stub):
    for make, prefix in ((_whole, "spec_verify_"), (_packed, "spec_verify_packed_")):
        cache = make()
        sv.paged_attention(torch.zeros(3, 4, 32, dtype=BF16), cache, torch.zeros(3, dtype=I64),
                           out=sv.AttentionOutputs.allocate(3, 4, 32, 3, device="cpu"))
        sv.kv_commit(cache, torch.zeros(4, dtype=I32), torch.zeros(6, dtype=I64), torch.zeros(6, dtype=I64), max_len=2)
        assert [c[0] for c in stub.calls[-2:]] == [prefix + ("attention" if make is _packed else "paged_attention"), prefix + "kv_commit"]


# ----------------------------------------------------------------------------------------------------------------------
# The library
# ----------------------------------------------------------------------------------------------------------------------

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, SMALL = 0, 1, 2, 3, 4, 5, 6
A = 1 << 32  # addresses that are never dereferenced


def _c_packed(**kw):
    f = dict(data=A, dtype=1, layers=2, pages=6, page_size=4, heads=2, head_dim=32, layer_stride=6 * 2 * 144, page_stride=2 * 144,
             head_stride=144, page_table=A << 4, max_pages=4, ld_table=4)
    f.update(kw)
    return sv.SvPackedKvCache(*[f[n] for n, _ in sv.SvPackedKvCache._fields_])


def _c_whole(**kw):
    f = dict(k=A, v=A + (1 << 24), dtype=1, layers=2, pages=6, page_size=4, heads=2, head_dim=32, layer_stride=6 * 4 * 64,
             page_stride=4 * 64, slot_stride=64, head_stride=32, page_table=A << 4, max_pages=4, ld_table=4)
    f.update(kw)
    return sv.SvKvCache(*[f[n] for n, _ in sv.SvKvCache._fields_])


def _c_append(lib, cache, rows=None, rot=None, **kw):
    r = dict(batch=3, max_len=2, total_rows=6, cu_seqlens=None, seq_lens=A << 5, row_slots=None)
    r.update(rows or {})
    t = dict(inv_freq=A << 6, pairs=16, interleaved=0, magnitude=1.0)
    t.update(rot or {})
    a = dict(layer=0, positions=None, k=A * 3, k_row=64, k_head=32, v=A * 5, v_row=64, v_head=32, q=A * 7, q_row=128, q_head=32,
             heads=4, out=A * 9, o_row=128, o_head=32, status=A << 7, rotation=True)
    a.update(kw)
    desc = sv.SvRows(*[r[n] for n, _ in sv.SvRows._fields_])
    rotation = sv.SvRotation(*[t[n] for n, _ in sv.SvRotation._fields_])
    fn = lib.spec_verify_packed_kv_append if isinstance(cache, sv.SvPackedKvCache) else lib.spec_verify_kv_append
    return fn(ctypes.byref(cache), a["layer"], ctypes.byref(desc), a["positions"], ctypes.byref(rotation) if a["rotation"] else None,
              a["k"], a["k_row"], a["k_head"], a["v"], a["v_row"], a["v_head"], a["q"], a["q_row"], a["q_head"], a["heads"],
              a["out"], a["o_row"], a["o_head"], a["status"], None)


@pytest.mark.parametrize("make", [_c_whole, _c_packed])
@pytest.mark.parametrize("kw,want", [
    (dict(rows=dict(batch=-1)), SHAPE), (dict(rows=dict(batch=65536)), SHAPE), (dict(rows=dict(max_len=0)), SHAPE),
    (dict(rows=dict(total_rows=5)), SHAPE), (dict(rows=dict(total_rows=1 << 31)), SHAPE), (dict(layer=2), SHAPE), (dict(layer=-1), SHAPE),
    (dict(rot=dict(pairs=17)), SHAPE), (dict(rot=dict(pairs=-1)), SHAPE), (dict(rot=dict(magnitude=float("nan"))), SHAPE),
    (dict(rot=dict(inv_freq=None)), NULL), (dict(heads=0), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL), (dict(out=None), NULL),
    (dict(status=None), NULL), (dict(rows=dict(seq_lens=None)), NULL),
    (dict(rows=dict(seq_lens=None, row_slots=A << 8)), NULL), (dict(k=A * 3 + 2), ALIGN), (dict(q_row=132), ALIGN),
    (dict(k_head=-32), SHAPE), (dict(o_row=0), UNSUPPORTED), (dict(o_head=16), UNSUPPORTED),
    (dict(out=A * 7 + 64), UNSUPPORTED), (dict(out=A * 3), UNSUPPORTED), (dict(out=A * 5 + 64), UNSUPPORTED),
    (dict(k=A), UNSUPPORTED), (dict(v=A + 64), UNSUPPORTED), (dict(out=A), UNSUPPORTED), (dict(q=A), UNSUPPORTED),
    (dict(rows=dict(batch=0)), OK), (dict(rows=dict(total_rows=0, cu_seqlens=A << 8)), OK)])
def test_library_refuses_appends(lib, make, kw, want):
    assert _c_append(lib, make(), **kw) == want


def test_library_refuses_caches(lib):
    for kw, want in ((dict(data=None), NULL), (dict(page_table=None), NULL), (dict(dtype=3), DTYPE), (dict(head_dim=48), SHAPE),
                     (dict(head_dim=288), SHAPE), (dict(page_size=0), SHAPE), (dict(heads=0), SHAPE), (dict(ld_table=3), SHAPE),
                     (dict(page_stride=-16), SHAPE), (dict(head_stride=152), ALIGN), (dict(data=A + 8), ALIGN),
                     (dict(head_stride=128), UNSUPPORTED), (dict(page_stride=144), UNSUPPORTED), (dict(layer_stride=0), UNSUPPORTED),
                     (dict(pages=1 << 29), SHAPE)):
        assert _c_append(lib, _c_packed(**kw)) == want, kw
        c = _c_packed(**kw)
        if want != UNSUPPORTED:
            assert lib.spec_verify_packed_attention(A, 128, 32, 4, ctypes.byref(c), 0, 3, 6, 2, None, A, None, None, 1.0, A, 128, 32, None,
                                                    A, A, 1 << 30, None) == want, kw
        assert lib.spec_verify_packed_kv_commit(ctypes.byref(c), 3, 2, 6, A, A, A, None, None) == want, kw
    for kw in (dict(slot_stride=0), dict(v=A + 64), dict(page_stride=128)):
        assert _c_append(lib, _c_whole(**kw)) == UNSUPPORTED, kw


def test_library_refuses_attention_and_commits(lib):
    c = _c_packed()
    attn = lambda cache=c, layer=0, batch=3, rows=6, heads=4, ws=A, size=1 << 30, q=A: lib.spec_verify_packed_attention(
        q, 128, 32, heads, ctypes.byref(cache), layer, batch, rows, 2, None, A, None, None, 1.0, A, 128, 32, None, A, ws, size, None)
    assert attn(cache=_c_packed(dtype=0)) == DTYPE and attn(layer=2) == SHAPE and attn(batch=4) == SHAPE and attn(heads=3) == SHAPE
    assert attn(ws=None) == SMALL and attn(size=100) == SMALL and attn(q=None) == NULL and attn(q=A + 2) == ALIGN and attn(batch=0) == OK
    commit = lambda max_len=2, n=6, cu=A, src=A: lib.spec_verify_packed_kv_commit(ctypes.byref(c), 3, max_len, n, cu, src, A, None, None)
    assert commit(max_len=0) == SHAPE and commit(max_len=1025) == SHAPE and commit(n=-1) == SHAPE and commit(cu=None) == NULL
    assert commit(src=None) == NULL


def test_library_refuses_reads(lib):
    def read(cache, layer=0, layers=1, k=A * 3, v=A * 5, ls=6 * 64, rs=64, hs=32, status=A << 7, **r):
        f = dict(batch=3, max_len=2, total_rows=6, cu_seqlens=None, seq_lens=A << 5, row_slots=None)
        f.update(r)
        desc = sv.SvRows(*[f[n] for n, _ in sv.SvRows._fields_])
        fn = lib.spec_verify_packed_kv_read if isinstance(cache, sv.SvPackedKvCache) else lib.spec_verify_kv_read
        return fn(ctypes.byref(cache), layer, layers, ctypes.byref(desc), k, v, ls, rs, hs, status, None)
    for c in (_c_whole(), _c_packed()):
        assert read(c, layer=1, layers=2) == SHAPE and read(c, layer=-1) == SHAPE and read(c, layers=-1) == SHAPE
        assert read(c, k=None) == NULL and read(c, status=None) == NULL and read(c, seq_lens=None) == NULL
        assert read(c, k=A * 3 + 4) == ALIGN and read(c, rs=68) == ALIGN and read(c, rs=-64) == SHAPE
        assert read(c, rs=32) == UNSUPPORTED and read(c, hs=0) == UNSUPPORTED and read(c, layers=2, ls=64) == UNSUPPORTED
        assert read(c, v=A * 3) == UNSUPPORTED and read(c, k=A) == UNSUPPORTED and read(c, v=A + 16) == UNSUPPORTED
        assert read(c, layers=0) == OK and read(c, batch=0, total_rows=0) == OK


def test_block_bytes(lib):
    for page in (1, 2, 3, 5, 16, 100, 128):
        for dim in range(32, 257, 32):
            assert sv.PackedKvCache.block_bytes(page, dim) == packed.block_bytes(page, dim)
    assert lib.spec_verify_packed_kv_block_bytes(16, 40) == 0 and lib.spec_verify_packed_kv_block_bytes(0, 64) == 0
    assert lib.spec_verify_packed_kv_block_bytes(16, 512) == 0


# ----------------------------------------------------------------------------------------------------------------------
# The oracle
# ----------------------------------------------------------------------------------------------------------------------


def test_the_formats_numbers():
    """Scales are half floats without their sign and lower mantissa bits; codes are e2m1."""
    bits = (np.arange(packed.MOST + 1, dtype=np.uint16) << 7).view(np.float16)
    assert np.array_equal(bits.astype(np.float64), packed.SCALES) and packed.SCALES[-1] == 10240
    for i, m in enumerate(packed.MAGNITUDES):
        e, f = i >> 1, i & 1
        assert m == (f * 0.5 if e == 0 else (1 + f * 0.5) * 2.0 ** (e - 1))


def test_quantising_is_nearest():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)) * 2.0 ** rng.integers(-20, 12, (200, 1))
    codes, scales, value = packed.quantize(x)
    assert np.array_equal(packed.values(codes, scales), value)
    s = packed.SCALES[scales].repeat(16, -1)
    grid = packed.MAGNITUDES * s[..., None]
    assert np.array_equal(np.abs(np.abs(x) - np.abs(value)), np.abs(np.abs(x)[..., None] - grid).min(-1))
    top = np.abs(x).reshape(200, 4, 16).max(-1)
    assert np.allclose(np.abs(6 * packed.SCALES[scales] - top), np.abs(6 * packed.SCALES - top[..., None]).min(-1))
    # what is held is held: quantising it again changes nothing
    again = packed.quantize(value)[2]
    full = (np.abs(value).reshape(200, 4, 16).max(-1) == 6 * packed.SCALES[scales]).repeat(16, -1)
    assert np.array_equal(again[full], value[full])


def test_blocks_and_back():
    rng = np.random.default_rng(1)
    for page, dim in ((1, 32), (5, 96), (16, 128)):
        parts = [rng.integers(0, 16, (2, 3, page, 2, dim)).astype(np.uint8), rng.integers(0, 256, (2, 3, page, 2, dim // 16)).astype(np.uint8),
                 rng.integers(0, 16, (2, 3, page, 2, dim)).astype(np.uint8), rng.integers(0, 256, (2, 3, page, 2, dim // 16)).astype(np.uint8)]
        b = packed.blocks(*parts)
        for a, c in zip(parts, packed.unblock(b, page, dim)):
            assert np.array_equal(a, c)
        # one entry by its bytes
        assert b[1, 2, 1, (page - 1) * (dim // 2) + 3] == parts[0][1, 2, page - 1, 1, 6] + 16 * parts[0][1, 2, page - 1, 1, 7]
        assert b[0, 1, 0, page * dim + page * (dim // 16) + 1] == parts[3][0, 1, 0, 0, 1]


def test_rotation_against_its_formula():
    rng = np.random.default_rng(2)
    x, f = rng.standard_normal((3, 2, 12)), rng.random(4)
    for inter in (False, True):
        y, _ = packed.rotate(x, [0, 5, -3], f, inter, 1.5)
        for r, pos in enumerate((0, 5, -3)):
            for i in range(4):
                a, b = (2 * i, 2 * i + 1) if inter else (i, i + 4)
                c, s = np.cos(pos * f[i]), np.sin(pos * f[i])
                assert np.allclose(y[r, :, a], 1.5 * (x[r, :, a] * c - x[r, :, b] * s))
                assert np.allclose(y[r, :, b], 1.5 * (x[r, :, b] * c + x[r, :, a] * s))
        assert np.array_equal(y[..., 8:], x[..., 8:])
        # products of queries and keys depend on the distance alone
        q, _ = packed.rotate(x[:1], [17], f, inter)
        k, _ = packed.rotate(x[1:2], [13], f, inter)
        q0, _ = packed.rotate(x[:1], [4], f, inter)
        assert np.allclose((q * k)[..., :8].sum(), (q0 * x[1:2])[..., :8].sum())


def test_angles_of_far_positions_against_rational_numbers():
    """Fewer whole turns by subtraction alone: the angle of n is twice that of n / 2, from one that fp64 holds exactly."""
    f = (10000.0 ** (-np.arange(8) / 8)).astype(np.float32)
    near = np.array([3, 2 ** 28 + 1, -(2 ** 28) - 7, 2 ** 29 - 1], np.int64)
    assert np.array_equal(packed.angles(near, f), near[:, None] * f.astype(np.float64))
    for p in near:
        z = np.exp(1j * packed.angles([p], f))
        for k in range(1, 33):
            z = z * z  # (twice the error each time)
            far = packed.angles([int(p) << k], f)
            assert (k < 3 or p == 3 or np.abs(far).max() <= np.pi) and np.abs(np.exp(1j * far) - z).max() <= 2.0 ** (k - 51)


def test_calls_run_on_their_tensors_device(monkeypatch):
    """Another device than the current one is entered and left again, a refused call's too; the current one is not touched."""
    now, moves = [1], []
    monkeypatch.setattr(sv, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "set_device", lambda d: (moves.append(d), now.__setitem__(0, d)))
    assert sv._run_on(1, lambda *a: (now[0], a), 5, 6) == (1, (5, 6)) and moves == []
    assert sv._run_on(0, lambda *a: (now[0], a), 7) == (0, (7,)) and moves == [0, 1]
    with pytest.raises(ctypes.ArgumentError):
        sv._run_on(0, sv.load_library().spec_verify_packed_kv_block_bytes, "16", 64)
    assert moves == [0, 1, 0, 1] and now == [1]
