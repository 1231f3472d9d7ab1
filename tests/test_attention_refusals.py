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
