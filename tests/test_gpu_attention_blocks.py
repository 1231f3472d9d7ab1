"""Attention of blocks of many rows, causal and under masks of any shape."""
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


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [127, 129, 257, 512, 1024])
@pytest.mark.parametrize("history", [0, 700])
def test_causal_blocks(dtype, rows, history):
    c = AttentionCase([history], rows, 2, 1, 64, 16, dtype, seed=rows + history)
    first = c.run(sv)
    check_attention(c, first)
    again = c.run(sv)
    assert torch.equal(first.out, again.out) and torch.equal(first.lse, again.lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [128, 256])
def test_causal_blocks_of_several_requests(dtype, dim):
    c = AttentionCase([130, 0, 64], [200, 300, 129], 4, 2, dim, 16, dtype, ragged=True, seed=dim)
    check_attention(c, c.run(sv))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [2, 3, 20, 130])
@pytest.mark.parametrize("shape", ["all", "upper", "random", "none"])
def test_masks_of_any_shape(dtype, rows, shape):
    # also rows that see later ones, and rows that do not see themselves
    c = AttentionCase([200, 0, 128], rows, 8, 2, 64, 16, dtype, tree=True, staged=True, seed=rows)
    rng = np.random.default_rng(rows)
    full = np.ones((3, rows, rows), np.uint8)
    c.mask = {"all": full, "upper": np.triu(full), "random": (rng.random(full.shape) < 0.4).astype(np.uint8) * 255,
              "none": 0 * full}[shape]
    check_attention(c, c.run(sv))
