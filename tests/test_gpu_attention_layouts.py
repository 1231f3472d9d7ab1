"""Attention over the paged cache against the fp64 oracle where the way K and V are brought in changes: page sizes with and
without whole boxes, histories that end anywhere in a page, wide heads, bad pages among good ones, many requests over
several cache heads; scales of either sign and zero; repeats."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from reject_row_vocab_gb300 import _build  # noqa: E402

_build.build()
from reject_row_vocab_gb300 import specverify as sv  # noqa: E402
from tests.serving_cases import BF16, F32, AttentionCase, check_attention  # noqa: E402

# the three ways of a kernel's rows: one token, a chain that shares a small unit, a block of many rows
ROWS = [1, 3, 18]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("page", [8, 16, 24, 40, 128, 256, 13])
def test_page_sizes_with_long_histories(dtype, rows, page):
    c = AttentionCase([517, 640, 263, 129], rows, 8, 2, 64, page, dtype, seed=page + rows)
    check_attention(c, c.run(sv))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("dim", [40, 96, 136, 192, 200, 256])
@pytest.mark.parametrize("page", [1, 16])
def test_head_sizes_with_long_histories(dtype, rows, dim, page):
    c = AttentionCase([400, 131], rows, 4, 2, dim, page, dtype, tree=rows > 1, staged=rows > 1, seed=dim + rows)
    check_attention(c, c.run(sv))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dim", [64, 256])
def test_bad_pages_among_good_ones(dtype, rows, page, dim):
    c = AttentionCase([700, 600, 300], rows, 8, 2, dim, page, dtype, seed=3 * page + rows)
    c.table[0, 2], c.table[0, 7] = -1, 10 ** 6
    c.table[2, 0] = -(1 << 31)
    got = c.run(sv)
    check_attention(c, got)
    assert got.dev_status.tolist() == [128, 0, 128]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 20])
def test_many_requests_over_several_cache_heads(dtype, rows):
    # more requests than a block has threads; some blocks begin in a later head, far into its requests
    lens = np.random.default_rng(rows).integers(0, 300, 600).tolist()
    c = AttentionCase(lens, rows, 3, 3, 64, 16, dtype, seed=rows)
    check_attention(c, c.run(sv))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-3])
def test_scales(dtype, rows, scale):
    c = AttentionCase([150, 0, 37], rows, 8, 2, 128, 16, dtype, tree=rows > 1, seed=rows)
    c.scale = scale
    check_attention(c, c.run(sv))


@pytest.mark.parametrize("dtype,dim,rows,page", [(BF16, 64, 2, 16), (BF16, 128, 4, 1), (BF16, 256, 1, 16), (BF16, 256, 20, 64),
                                                 (BF16, 256, 40, 5), (F32, 64, 12, 16), (F32, 200, 3, 16), (F32, 256, 2, 1)])
def test_repeats_are_bit_equal(dtype, dim, rows, page):
    c = AttentionCase([9001, 130, 0, 2500], rows, 4, 1, dim, page, dtype, seed=dim)
    first = c.run(sv)
    check_attention(c, first)
    for _ in range(8):
        again = c.run(sv)
        assert torch.equal(first.out, again.out) and torch.equal(first.lse, again.lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("axis", ["pages", "heads"])
def test_entries_that_share_their_memory(dtype, rows, axis):
    # one page, or one head, repeated without a step
    c = AttentionCase([300, 170], rows, 4, 2, 64, 16, dtype, seed=rows, poison=False)
    one = (slice(None), slice(0, 1)) if axis == "pages" else (slice(None), slice(None), slice(None), slice(0, 1))
    shape = c.k.shape
    c.k, c.v = c.k[one].contiguous().expand(shape), c.v[one].contiguous().expand(shape)
    k, v = c.k[one].cuda().expand(shape), c.v[one].cuda().expand(shape)
    assert 0 in k.stride()
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    cache = sv.PagedKvCache(k, v, dev(c.table))
    got = sv.paged_attention(c.q.cuda(), cache, dev(np.asarray(c.lens, np.int64)), max_len=c.max_len, scale=c.scale)
    check_attention(c, got)
