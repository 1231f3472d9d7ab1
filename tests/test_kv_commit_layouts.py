"""Caches that the KV commit refuses (no GPU): entries, heads, layers, or K and V, that share memory.  Their moves would be
made several times and in no order."""
import ctypes

import pytest

pytest.importorskip("torch")

from reject_row_vocab_gb300 import specverify as sv  # noqa: E402
from tests.test_serving_checks import FAKE, UNSUPPORTED, _struct, lib  # noqa: E402,F401

APART = 1 << 30  # bytes between K and V
LAYER, PAGE, SLOT, HEAD = 2 * (1 << 20), 2 * 2048, 2 * 128, 2 * 64  # bytes of the steps of _struct


@pytest.mark.parametrize("kw", [
    dict(head_stride=0), dict(slot_stride=0), dict(page_stride=0), dict(layer_stride=0),   # repeated without a step
    dict(head_stride=32), dict(slot_stride=64), dict(page_stride=1024), dict(layer_stride=8 * 2048 - 8),  # steps too short
    dict(slot_stride=128, head_stride=128 * 16, page_stride=2048),  # head-major pages that lie over one another
    dict(v=FAKE), dict(v=FAKE + 16), dict(v=FAKE + HEAD), dict(v=FAKE + SLOT), dict(v=FAKE + 3 * PAGE), dict(v=FAKE + LAYER),
    dict(v=FAKE + LAYER - PAGE), dict(v=FAKE - 16), dict(v=FAKE - LAYER - 7 * PAGE - 15 * SLOT - HEAD),
    dict(layers=1, v=FAKE + 8 * PAGE - 16)])
def test_shared_memory_is_refused(lib, kw):  # noqa: F811
    kw.setdefault("v", FAKE + APART)
    assert lib.spec_verify_kv_commit(ctypes.byref(_struct(**kw)), 1, 4, 4, FAKE, FAKE, FAKE, None, None) == UNSUPPORTED


def test_the_error_says_so():
    assert sv.STATUS[UNSUPPORTED] == "SV_ERR_UNSUPPORTED"
