"""The KV move in caches whose K and V lie in one another's gaps, against the oracle; and the refusal of caches whose entries
share memory, which comes before anything is enqueued."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from oracle import serving  # noqa: E402
from reject_row_vocab_gb300 import _build  # noqa: E402

_build.build()
from reject_row_vocab_gb300 import specverify as sv  # noqa: E402

L, P, S, H, D = 3, 20, 16, 4, 64


def _lists(n=3):
    table = np.random.default_rng(1).permutation(P)[:9].reshape(n, 3)
    src = [int(table[b, 1]) * S + j for b in range(n) for j in (0, 2, 5, 9)]
    dst = [S + j for _ in range(n) for j in range(4)]
    return table, [0, 4, 8, 12], src, dst


def _run(k, v):
    table, cu, src, dst = _lists()
    up = lambda a, t: torch.tensor(np.asarray(a), dtype=t).cuda()  # noqa: E731
    return sv.kv_commit(sv.PagedKvCache(k, v, up(table, torch.int32)), up(cu, torch.int32), up(src, torch.int64),
                        up(dst, torch.int64), max_len=4)


def _store(*shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("kv", [
    lambda: _store(2, L, P, S, H, D).unbind(0), lambda: _store(L, 2, P, S, H, D).unbind(1),
    lambda: _store(L, P, 2, S, H, D).unbind(2), lambda: _store(L, P, S, 2, H, D).unbind(3),
    lambda: _store(L, P, S, H, 2, D).unbind(4), lambda: _store(L, P, S, H, 2 * D).chunk(2, -1),
    lambda: tuple(x.transpose(2, 3) for x in _store(L, P, 2, H, S, D).unbind(2)),
    lambda: (lambda x: (x[0:2 * L:2], x[5:5 + 2 * L:2]))(_store(2 * L + 5, P, S, H, D))])
def test_interleaved_caches(kv):
    k, v = kv()
    before = [x.float().cpu().contiguous().numpy() for x in (k, v)]  # (the oracle goes over a dense array)
    assert _run(k, v).tolist() == [0, 0, 0]
    table, cu, src, dst = _lists()
    for mine, was in zip((k, v), before):
        assert np.array_equal(mine.float().cpu().numpy(), serving.kv_commit(was, table, cu, src, dst, 4)[0])


@pytest.mark.parametrize("kv", [
    lambda: [_store(L, P, S, H, D)] * 2,
    lambda: [_store(L, P, S, 1, D).expand(L, P, S, H, D) for _ in range(2)],
    lambda: [_store(1, P, S, H, D).expand(L, P, S, H, D) for _ in range(2)],
    lambda: (lambda x: (x[:L], x[1:]))(_store(L + 1, P, S, H, D))])
def test_shared_memory_is_refused(kv):
    k, v = kv()
    before = k.clone(), v.clone()
    with pytest.raises(sv.SpecVerifyError) as e:
        _run(k, v)
    assert e.value.code == 5
    assert torch.equal(k, before[0]) and torch.equal(v, before[1])
