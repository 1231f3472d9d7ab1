"""Refusals of the serving-side operators (no GPU): the binding's argument checks, run on CPU tensors with the library's
entry points replaced by stubs, and the library's own checks, which come before anything is enqueued.  And the fp64 oracle
against direct formulas and differences."""
import ctypes
import os
import sys

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from oracle import serving  # noqa: E402
from reject_row_vocab_gb300 import specverify as sv  # noqa: E402
from tests.serving_cases import random_tree  # noqa: E402

ENTRY = ("spec_verify_paged_attention", "spec_verify_kv_commit", "spec_verify_token_logprobs",
         "spec_verify_token_logprobs_backward")
BF16, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


class _StubLib:
    """The real library for sizes; the entry points only record their calls."""

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
def cpu_binding(lib, monkeypatch):
    stub = _StubLib(lib)
    monkeypatch.setattr(sv, "load_library", lambda: stub)
    monkeypatch.setattr(sv, "_call_stream", lambda s, d: None)
    monkeypatch.setattr(sv, "_require_cuda", lambda t, name="logits": None)
    monkeypatch.setattr(sv, "_require_cache", lambda c: None)
    return stub


# ----------------------------------------------------------------------------------------------------------------------
# The binding
# ----------------------------------------------------------------------------------------------------------------------


def _kv(layers=2, pages=6, page=4, heads=2, dim=16, dtype=BF16):
    return torch.zeros(layers, pages, page, heads, dim, dtype=dtype)


def _cache(**kw):
    return sv.PagedKvCache(_kv(**kw), _kv(**kw), torch.zeros(3, 4, dtype=I32))


def _attn(**kw):
    a = dict(q=torch.zeros(6, 4, 16, dtype=BF16), cache=_cache(), seq_lens=torch.zeros(3, dtype=I64), max_len=2)
    a.update(kw)
    if "ws" not in a:
        a["ws"] = sv.attention_workspace(3, 2, a["cache"], 4)
    return sv.paged_attention(a.pop("q"), a.pop("cache"), a.pop("seq_lens"), **a)


@pytest.mark.parametrize("good", [
    dict(), dict(max_len=None), dict(mask=torch.zeros(3, 2, 2, dtype=torch.uint8)), dict(scale=0.0), dict(layer=1),
    dict(row_slots=torch.zeros(6, dtype=I64)), dict(cu_seqlens=torch.zeros(4, dtype=I32)),
    dict(q=torch.zeros(6, 8, 32, dtype=BF16)[:, ::2, :16]), dict(seq_lens=torch.zeros(0, dtype=I64), max_len=1),
    dict(out=sv.AttentionOutputs.allocate(6, 4, 16, 3, device="cpu", lse=False))])
def test_attention_passes_what_it_takes(cpu_binding, good):
    _attn(**good)
    assert [c[0] for c in cpu_binding.calls] == ["spec_verify_paged_attention"]


def test_attention_hands_on_strides_and_scale(cpu_binding):
    q = torch.zeros(6, 8, 32, dtype=BF16)[:, ::2, :16]
    _attn(q=q, scale=0.25, layer=1)
    a = cpu_binding.calls[0][1]
    assert a[:4] == (q.data_ptr(), 256, 64, 4) and a[5:9] == (1, 3, 6, 2) and a[13] == 0.25


@pytest.mark.parametrize("bad", [
    dict(q=torch.zeros(6, 64, dtype=BF16)), dict(q=torch.zeros(6, 4, 16)), dict(q=torch.zeros(6, 4, 8, dtype=BF16)),
    dict(q=torch.zeros(6, 4, 32, dtype=BF16)[:, :, ::2]), dict(q=torch.zeros(5, 4, 16, dtype=BF16)),
    dict(seq_lens=None), dict(seq_lens=torch.zeros(3, dtype=I32)), dict(seq_lens=torch.zeros(4, dtype=I64)),
    dict(seq_lens=torch.zeros(6, dtype=I64)[::2]), dict(cu_seqlens=torch.zeros(3, dtype=I32)),
    dict(cu_seqlens=torch.zeros(4, dtype=I64)), dict(cu_seqlens=torch.zeros(4, dtype=I32), max_len=None),
    dict(row_slots=torch.zeros(5, dtype=I64)), dict(row_slots=torch.zeros(6, dtype=I32)),
    dict(mask=torch.zeros(3, 2, 1, dtype=torch.uint8)), dict(mask=torch.zeros(3, 2, 2, dtype=torch.bool)),
    dict(ws=torch.zeros(1 << 20, dtype=F32)),
    dict(out=sv.AttentionOutputs.allocate(5, 4, 16, 3, device="cpu")),
    dict(out=sv.AttentionOutputs.allocate(6, 4, 16, 3, dtype=F32, device="cpu")),
    dict(out=sv.AttentionOutputs.allocate(6, 4, 16, 2, device="cpu"))])
def test_attention_refuses(cpu_binding, bad):
    with pytest.raises((TypeError, ValueError)):
        _attn(**bad)
    assert cpu_binding.calls == []


@pytest.mark.parametrize("k,v,table", [
    (_kv()[0], _kv()[0], None), (_kv(dtype=torch.float16), _kv(dtype=torch.float16), None), (_kv(), _kv(dtype=F32), None),
    (_kv(), _kv(pages=5), None), (_kv(), _kv(heads=4)[:, :, :, ::2], None), (_kv(dim=32)[..., ::2], _kv(dim=32)[..., ::2], None),
    (_kv(), _kv(), torch.zeros(3, 4, dtype=I64)), (_kv(), _kv(), torch.zeros(12, dtype=I32)),
    (_kv(), _kv(), torch.zeros(3, 8, dtype=I32)[:, ::2])])
def test_cache_refuses(k, v, table):
    with pytest.raises((TypeError, ValueError)):
        sv.PagedKvCache(k, v, torch.zeros(3, 4, dtype=I32) if table is None else table)


def test_a_cache_on_the_host_is_refused(lib):
    with pytest.raises(ValueError):
        _attn()
    with pytest.raises(ValueError):
        sv.kv_commit(_cache(), torch.zeros(4, dtype=I32), torch.zeros(3, dtype=I64), torch.zeros(3, dtype=I64), max_len=1)
    with pytest.raises((TypeError, ValueError)):
        sv.kv_commit(None, torch.zeros(4, dtype=I32), torch.zeros(3, dtype=I64), torch.zeros(3, dtype=I64), max_len=1)
    with pytest.raises(ValueError):
        sv.token_logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=I32))


def _commit(**kw):
    a = dict(cu=torch.zeros(4, dtype=I32), src=torch.zeros(3, dtype=I64), dst=torch.zeros(3, dtype=I64), max_len=2)
    a.update(kw)
    return sv.kv_commit(_cache(), a.pop("cu"), a.pop("src"), a.pop("dst"), **a)


def test_commit_passes_what_it_takes(cpu_binding):
    _commit()
    _commit(src=torch.zeros(0, dtype=I64), dst=torch.zeros(5, dtype=I64))
    assert [c[1][1:4] for c in cpu_binding.calls] == [(3, 2, 3), (3, 2, 0)]


@pytest.mark.parametrize("bad", [
    dict(cu=None), dict(cu=torch.zeros(4, dtype=I64)), dict(cu=torch.zeros(0, dtype=I32)), dict(cu=torch.zeros(5, dtype=I32)),
    dict(src=None), dict(dst=torch.zeros(3, dtype=I32)), dict(src=torch.zeros(6, dtype=I64)[::2]),
    dict(dev_status=torch.zeros(2, dtype=I32)), dict(dev_status=torch.zeros(3, dtype=I64))])
def test_commit_refuses(cpu_binding, bad):
    with pytest.raises((TypeError, ValueError)):
        _commit(**bad)
    assert cpu_binding.calls == []


def _logp(**kw):
    a = dict(logits=torch.zeros(4, 16), ids=torch.zeros(4, 2, dtype=I32), top_k=3)
    a.update(kw)
    if "ws" not in a:
        a["ws"] = sv.logprobs_workspace(4, 16, 3, "cpu")
    return sv.token_logprobs(a.pop("logits"), a.pop("ids"), **a)


@pytest.mark.parametrize("good", [
    dict(), dict(ids=torch.zeros(4, dtype=I32)), dict(ids=torch.zeros(4, 5, dtype=I32)[:, 1:3]), dict(row_temp=torch.ones(4)),
    dict(ids=torch.zeros(4, 0, dtype=I32)), dict(row_index=torch.zeros(2, dtype=I32), ids=torch.zeros(2, dtype=I32)),
    dict(logits=torch.zeros(4, 24, dtype=BF16)[:, :15])])
def test_logprobs_pass_what_they_take(cpu_binding, good):
    _logp(**good)
    assert [c[0] for c in cpu_binding.calls] == ["spec_verify_token_logprobs"]


@pytest.mark.parametrize("bad", [
    dict(ids=None), dict(ids=torch.zeros(4, 2, dtype=I64)), dict(ids=torch.zeros(3, 2, dtype=I32)),
    dict(ids=torch.zeros(4, 4, dtype=I32)[:, ::2]), dict(ids=torch.zeros(4, 2, 1, dtype=I32)),
    dict(row_temp=torch.ones(3)), dict(row_temp=torch.ones(4, dtype=torch.float64)),
    dict(row_index=torch.zeros(5, dtype=I32)), dict(row_index=torch.zeros(4, dtype=I64)), dict(ws=torch.zeros(4096)),
    dict(logits=torch.zeros(4, 16, dtype=torch.float16)),
    dict(out=sv.LogprobOutputs.allocate(3, 2, 3, "cpu")), dict(out=sv.LogprobOutputs.allocate(4, 1, 3, "cpu")),
    dict(out=sv.LogprobOutputs.allocate(4, 2, 2, "cpu"))])
def test_logprobs_refuse(cpu_binding, bad):
    with pytest.raises((TypeError, ValueError)):
        _logp(**bad)
    assert cpu_binding.calls == []


def _grad(**kw):
    a = dict(logits=torch.zeros(4, 16), ids=torch.zeros(4, 2, dtype=I32), kept=sv.LogprobOutputs.allocate(4, 2, 3, "cpu"),
             g=torch.zeros(4, 2))
    a.update(kw)
    return sv.token_logprobs_backward(a.pop("logits"), a.pop("ids"), a.pop("kept"), a.pop("g"), **a)


def test_gradient_passes_what_it_takes(cpu_binding):
    _grad()
    _grad(g_entropy=torch.zeros(4), g_top=torch.zeros(4, 3), row_temp=torch.ones(4))
    _grad(out=torch.zeros(4, 32)[:, :16])
    assert len(cpu_binding.calls) == 3


@pytest.mark.parametrize("bad", [
    dict(g=torch.zeros(4, 1)), dict(g=torch.zeros(4, 2, dtype=torch.float64)), dict(g_entropy=torch.zeros(3)),
    dict(g_top=torch.zeros(12)), dict(g_top=torch.zeros(4, 2)), dict(row_temp=torch.ones(3)),
    dict(kept=sv.LogprobOutputs.allocate(3, 2, 3, "cpu")), dict(out=torch.zeros(4, 15)), dict(out=torch.zeros(3, 16)),
    dict(out=torch.zeros(4, 16, dtype=BF16)), dict(ids=torch.zeros(4, 2, dtype=I64))])
def test_gradient_refuses(cpu_binding, bad):
    with pytest.raises((TypeError, ValueError)):
        _grad(**bad)
    assert cpu_binding.calls == []


# ----------------------------------------------------------------------------------------------------------------------
# The library
# ----------------------------------------------------------------------------------------------------------------------

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, SMALL = range(7)
FAKE = 0x100000  # aligned, never dereferenced on the host


def _struct(**kw):
    a = dict(k=FAKE, v=FAKE, dtype=sv.SV_BF16, layers=2, pages=8, page_size=16, heads=2, head_dim=64, layer_stride=1 << 20,
             page_stride=2048, slot_stride=128, head_stride=64, page_table=FAKE, max_pages=4, ld_table=4)
    a.update(kw)
    return sv.SvKvCache(*[a[n] for n, _ in sv.SvKvCache._fields_])


BAD_CACHES = [
    (dict(k=None), NULL), (dict(page_table=None), NULL), (dict(dtype=7), DTYPE), (dict(pages=0), SHAPE),
    (dict(page_size=0), SHAPE), (dict(heads=0), SHAPE), (dict(head_dim=264), SHAPE), (dict(head_dim=0), SHAPE),
    (dict(ld_table=3), SHAPE), (dict(slot_stride=-128), SHAPE), (dict(pages=1 << 20, page_size=1 << 12), SHAPE),
    (dict(k=FAKE + 8), ALIGN), (dict(head_dim=60), ALIGN), (dict(slot_stride=132), ALIGN)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_library_refuses_bad_caches(lib, kw, code):
    assert _attention(lib, cache=_struct(**kw)) == code
    assert lib.spec_verify_kv_commit(ctypes.byref(_struct(**kw)), 1, 4, 4, FAKE, FAKE, FAKE, None, None) == code


def _attention(lib, **kw):
    a = dict(q=FAKE, q_row=256, q_head=64, heads=4, cache=_struct(), layer=0, batch=2, rows=8, max_len=4, cu=None, lens=FAKE,
             slots=None, mask=None, scale=1.0, out=FAKE, o_row=256, o_head=64, lse=None, status=FAKE, ws=FAKE, ws_bytes=1 << 34)
    a.update(kw)
    a["cache"] = ctypes.byref(a["cache"]) if a["cache"] else None
    return lib.spec_verify_paged_attention(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(cache=None), NULL), (dict(q=None), NULL), (dict(out=None), NULL), (dict(lens=None), NULL), (dict(status=None), NULL),
    (dict(layer=2), SHAPE), (dict(layer=-1), SHAPE), (dict(batch=-1), SHAPE), (dict(batch=65536, rows=1 << 20), SHAPE),
    (dict(max_len=0), SHAPE), (dict(rows=7), SHAPE), (dict(heads=3), SHAPE), (dict(heads=0), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(q_row=-256), SHAPE),
    (dict(max_len=1 << 23, cu=FAKE), SHAPE), (dict(o_head=32), SHAPE), (dict(o_row=32), SHAPE),
    (dict(q=FAKE + 8), ALIGN), (dict(q_head=68), ALIGN), (dict(out=FAKE + 8), ALIGN), (dict(o_row=260), ALIGN),
    (dict(ws=None), SMALL), (dict(ws_bytes=1024), SMALL), (dict(ws=FAKE + 128), SMALL), (dict(batch=0), OK)])
def test_library_refuses_attention(lib, kw, code):
    assert _attention(lib, **kw) == code


def _lists(lib, **kw):
    a = dict(cache=ctypes.byref(_struct()), batch=2, max_len=4, n=8, cu=FAKE, src=FAKE, dst=FAKE, status=None)
    a.update(kw)
    return lib.spec_verify_kv_commit(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(cache=None), NULL), (dict(cu=None), NULL), (dict(src=None), NULL), (dict(dst=None), NULL), (dict(batch=-1), SHAPE),
    (dict(max_len=0), SHAPE), (dict(max_len=1025), SHAPE), (dict(n=-1), SHAPE), (dict(batch=0), OK)])
def test_library_refuses_commits(lib, kw, code):
    assert _lists(lib, **kw) == code


def _forward(lib, **kw):
    a = dict(logits=FAKE, dtype=sv.SV_F32, ld=64, rows=4, vocab=64, n=4, index=None, ids=FAKE, num=2, ldi=2, temp=None, top=3,
             logprob=FAKE, entropy=None, row_max=None, log_z=None, top_ids=FAKE, top_logprob=FAKE, flags=None, ws=FAKE,
             ws_bytes=1 << 34)
    a.update(kw)
    return lib.spec_verify_token_logprobs(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(logprob=None), NULL), (dict(top_ids=None), NULL),
    (dict(dtype=5), DTYPE), (dict(ld=32), SHAPE), (dict(vocab=0), SHAPE), (dict(rows=-1), SHAPE), (dict(n=-1), SHAPE),
    (dict(num=1025, ldi=1025), SHAPE), (dict(top=65), SHAPE), (dict(top=-1), SHAPE), (dict(ldi=1), SHAPE), (dict(n=5), SHAPE),
    (dict(logits=FAKE + 4), ALIGN), (dict(ld=66), ALIGN), (dict(ws=None), SMALL), (dict(ws_bytes=16), SMALL), (dict(n=0), OK)])
def test_library_refuses_logprobs(lib, kw, code):
    assert _forward(lib, **kw) == code


def _backward(lib, **kw):
    a = dict(logits=FAKE, dtype=sv.SV_F32, ld=64, rows=4, vocab=64, ids=FAKE, num=2, ldi=2, temp=None, row_max=FAKE, log_z=FAKE,
             entropy=None, top_ids=None, top=0, g=FAKE, g_entropy=None, g_top=None, out=2 * FAKE, ldd=64)
    a.update(kw)
    return lib.spec_verify_token_logprobs_backward(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), NULL), (dict(out=None), NULL), (dict(row_max=None), NULL), (dict(log_z=None), NULL), (dict(ids=None), NULL),
    (dict(g=None), NULL), (dict(g_entropy=FAKE), NULL), (dict(top=3, g_top=FAKE), NULL), (dict(dtype=5), DTYPE),
    (dict(ldd=32), SHAPE), (dict(ld=32), SHAPE), (dict(num=-1), SHAPE), (dict(top=65), SHAPE), (dict(out=2 * FAKE + 4), ALIGN),
    (dict(ldd=66), ALIGN), (dict(out=FAKE), UNSUPPORTED), (dict(out=FAKE + 512), UNSUPPORTED), (dict(rows=0), OK)])
def test_library_refuses_gradients(lib, kw, code):
    assert _backward(lib, **kw) == code


# ----------------------------------------------------------------------------------------------------------------------
# The oracle
# ----------------------------------------------------------------------------------------------------------------------


def test_oracle_attention_against_a_dense_softmax():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 1, 5, 4, 2, 8))[:, 0], rng.standard_normal((1, 5, 4, 2, 8))[0]
    k = k[0]
    table, L, n = np.array([[3, 1, 4]]), 6, 4
    q, mask = rng.standard_normal((n, 4, 8)), random_tree(rng, n)[1]
    r = serving.attention(q, k, v, table, [L], [0], [n], 0.3, mask=mask[None])
    slots = [table[0, x // 4] * 4 + x % 4 for x in range(L + n)]
    see = np.concatenate([np.ones((n, L), bool), mask.astype(bool)], 1)
    for h in range(4):
        s = np.where(see, q[:, h] @ k.reshape(20, 2, 8)[slots, h // 2].T * 0.3, -np.inf)
        e = np.exp(s)
        np.testing.assert_allclose(r["out"][:, h], e / e.sum(1, keepdims=True) @ v.reshape(20, 2, 8)[slots, h // 2], rtol=1e-12)
        np.testing.assert_allclose(r["lse"][:, h], np.log(e.sum(1)), rtol=1e-12)


def test_oracle_commit_reads_before_it_writes():
    a = np.arange(8.0).reshape(1, 2, 4, 1, 1)
    got, status = serving.kv_commit(a, np.array([[1, 0]]), [0, 3], [4, 5, 7], [1, 0, 2], 3)
    # positions 0, 1, 2 are slots 4, 5, 6; the entries are values 4, 5, 7
    assert got.ravel().tolist() == [0, 1, 2, 3, 5, 4, 7, 7] and status.tolist() == [0]


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(1)
    V, J, K, h = 9, 3, 4, 1e-5
    x, temp = rng.standard_normal((2, V)), np.array([0.7, 1.9])
    ids = np.array([[2, 2, -1], [8, 40, 0]])
    g, ge, gt = rng.standard_normal((2, J)), rng.standard_normal(2), rng.standard_normal((2, K))
    top = serving.logprobs(x, ids, temp, K)["top_ids"]

    def loss(y):
        lp = np.log(np.exp(y / temp[:, None]) / np.exp(y / temp[:, None]).sum(1, keepdims=True))
        total = (ge * -(np.exp(lp) * lp).sum(1)).sum() + sum(gt[i, k] * lp[i, top[i, k]] for i in range(2) for k in range(K))
        return total + sum(g[i, j] * lp[i, ids[i, j]] for i in range(2) for j in range(J) if 0 <= ids[i, j] < V)

    d, _ = serving.logprobs_grad(x, ids, g, temp, ge, top, gt)
    for i in range(2):
        for v in range(V):
            e = np.zeros_like(x)
            e[i, v] = h
            # a central difference's error: third derivatives of order 10 times h^2, and 1e-15 / h
            assert abs((loss(x + e) - loss(x - e)) / (2 * h) - d[i, v]) < 1e-8
