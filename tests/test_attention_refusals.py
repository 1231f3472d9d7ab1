"""Refusals of the attention call that depend on several arguments at once (no GPU)."""
import pytest

torch = pytest.importorskip("torch")

from reject_row_vocab_gb300 import specverify as sv  # noqa: E402
from tests.test_serving_checks import BF16, FAKE, SHAPE, _attention, _attn, cpu_binding, lib  # noqa: E402,F401


@pytest.mark.parametrize("kw", [
    dict(o_row=64, o_head=64), dict(o_row=128, o_head=64), dict(o_row=192, o_head=64), dict(o_row=248, o_head=64),
    dict(o_row=64, o_head=448), dict(o_row=128, o_head=64 * 14), dict(o_row=0, o_head=64), dict(o_row=256, o_head=0),
    dict(o_row=256, o_head=128)])
def test_outputs_that_lie_over_one_another(lib, kw):  # noqa: F811
    # 8 rows of 4 heads of 64: rows of heads, or heads of rows, each behind the other
    assert _attention(lib, **kw) == SHAPE


@pytest.mark.parametrize("kw", [dict(o_row=256, o_head=64), dict(o_row=264, o_head=64), dict(o_row=64, o_head=512), dict(o_row=128, o_head=64 * 15),
                                dict(o_row=512, o_head=64), dict(o_row=72, o_head=72 * 8)])
def test_outputs_beside_one_another(lib, kw):  # noqa: F811
    assert _attention(lib, batch=0, **kw) == 0


def test_a_binding_passes_overlapping_outputs_on_to_the_library(cpu_binding):  # noqa: F811
    buf = torch.zeros(1024, dtype=BF16)
    out = sv.AttentionOutputs.allocate(6, 4, 16, 3, device="cpu")
    out.out = buf.as_strided((6, 4, 16), (16, 16, 1))
    _attn(out=out)
    assert cpu_binding.calls[0][1][15:17] == (16, 16)


@pytest.mark.parametrize("rows", [4, 5, 7, 2])
def test_rows_that_no_request_would_own(cpu_binding, rows):  # noqa: F811
    # three requests and no max_len: the rows have to divide among them
    q = torch.zeros(rows, 4, 16, dtype=BF16)
    with pytest.raises(ValueError, match="max_len"):
        _attn(q=q, max_len=None)
    assert cpu_binding.calls == []


def test_rows_left_over_on_purpose(cpu_binding):  # noqa: F811
    _attn(q=torch.zeros(7, 4, 16, dtype=BF16), max_len=2)
    _attn(q=torch.zeros(9, 4, 16, dtype=BF16), max_len=None)
    assert [c[1][8] for c in cpu_binding.calls] == [2, 3]
