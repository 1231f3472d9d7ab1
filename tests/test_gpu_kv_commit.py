"""The KV move of the commit lists against the oracle, exactly."""
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


def _run(layers, pages, page, heads, dim, dtype, table, cu, src, dst, max_len, head_major=False):
    g = torch.Generator().manual_seed(pages + dim)
    k, v = (torch.randn(layers, pages, page, heads, dim, generator=g).to(dtype) for _ in range(2))
    lay = lambda t: t.cuda().transpose(2, 3).contiguous().transpose(2, 3) if head_major else t.cuda()
    dk, dv = lay(k), lay(v)
    up = lambda a, t: torch.tensor(a, dtype=t).cuda()
    cache = sv.PagedKvCache(dk, dv, up(table, torch.int32))
    st = sv.kv_commit(cache, up(cu, torch.int32), up(src, torch.int64), up(dst, torch.int64), max_len=max_len)
    for mine, host in ((dk, k), (dv, v)):
        want, status = serving.kv_commit(host.float().numpy(), np.asarray(table), cu, src, dst, max_len)
        assert np.array_equal(mine.float().cpu().numpy(), want)
        assert np.array_equal(st.cpu().numpy().view(np.uint32), status)
    return st


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads,dim,page", [(1, 8, 1), (8, 128, 16), (3, 80, 5), (2, 256, 64)])
@pytest.mark.parametrize("head_major", [False, True])
def test_staged_rows(dtype, heads, dim, page, head_major):
    rng = np.random.default_rng(dim + page)
    B, n, need = 5, 6, -(-40 // page)
    pages = B * need + -(-B * n // page)
    order = rng.permutation(pages)
    table = order[:B * need].reshape(B, need)
    slots = np.concatenate([p * page + np.arange(page) for p in order[B * need:]])[:B * n].reshape(B, n)
    cu, src, dst = [0], [], []
    for b in range(B):
        a = int(rng.integers(0, n + 1))
        src += slots[b][np.sort(rng.choice(n, a, replace=False))].tolist()
        dst += list(range(20 + b, 20 + b + a))
        cu.append(cu[-1] + a)
    _run(3, pages, page, heads, dim, dtype, table.tolist(), cu, src, dst, n, head_major)


@pytest.mark.parametrize("n", [1, 2, 17, 64, 300, 1024])
def test_rows_staged_in_place_overlap(n):
    # positions 10 .. 10 + n - 1 hold the new rows; the accepted ones move towards the front, in one call
    rng = np.random.default_rng(n)
    page = 16
    need = -(-(10 + n) // page)
    table = rng.permutation(need)[None]
    keep = [0] + sorted(rng.choice(np.arange(1, n), (n - 1) // 2, replace=False).tolist()) if n > 1 else [0]
    slot = lambda x: int(table[0, x // page]) * page + x % page
    src = [slot(10 + j) for j in keep]
    dst = [10 + i for i in range(len(keep))]
    _run(2, need, page, 4, 64, torch.bfloat16, table.tolist(), [0, len(keep)], src, dst, n)


def test_any_permutation_within_a_request():
    # reads come before writes: a reversal is a reversal, not a smear
    n, page = 200, 16
    need = -(-n // page)
    table = np.arange(need)[None]
    _run(1, need, page, 2, 64, torch.float32, table.tolist(), [0, n], list(range(n))[::-1], list(range(n)), n)


def test_bad_entries_and_ranges():
    table = [[0, 1], [2, -1], [3, 99], [4, 5], [6, 7]]
    cu = [0, 3, 6, 8, 7, 12]
    src = [70, 71, -1, 72, 73, 74, 75, 76, 77, 78, 79, 10 ** 12]
    dst = [0, 1, 2, 3, 40, 15, 16, -1, 3, 4, 5, 6]
    st = _run(2, 8, 16, 2, 64, torch.bfloat16, table, cu, src, dst, 4)
    assert st.tolist() == [128, 128, 128, 8, 8]


def test_nothing_to_commit():
    _run(1, 4, 16, 2, 64, torch.bfloat16, [[0], [1]], [0, 0, 0], [], [], 4)
