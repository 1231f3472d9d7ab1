"""Attention where K and V reach shared memory by turns in boxes and row by row, and where the values of new rows are taken
out of V: what one tile leaves must not reach the next."""
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


def _lens(n, seed):
    """Histories that end on a tile's edge, just behind it and within a page, with long ones in between."""
    rng = np.random.default_rng(seed)
    kinds = [lambda: int(rng.integers(0, 130)), lambda: 128 * int(rng.integers(1, 5)), lambda: 128 * int(rng.integers(1, 4)) + 1,
             lambda: int(rng.integers(500, 900))]
    return [kinds[i % 4]() for i in range(n)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 3, 18])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_boxes_where_gathered_rows_were(dtype, rows, dim):
    # about six requests a block: every place of the ring is taken by boxes and by gathered rows in turn
    c = AttentionCase(_lens(120, rows), rows, 8, 8, dim, 16, dtype, seed=dim)
    first = c.run(sv)
    for _ in range(3):
        again = c.run(sv)
        assert torch.equal(first.out, again.out) and torch.equal(first.lse, again.lse)
    # (the oracle goes key by key: a part of the requests)
    small = AttentionCase(_lens(24, rows), rows, 4, 2, dim, 16, dtype, seed=dim + 1)
    check_attention(small, small.run(sv))
