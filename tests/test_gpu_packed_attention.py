"""Attention over the 4-bit cache against the fp64 oracle on the values that the cache stands for."""
import numpy as np
import pytest
import torch

from oracle import packed
from tests.packed_cases import PackedAttentionCase
from tests.serving_cases import BF16, AttentionCase, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    from reject_row_vocab_gb300 import specverify
    return specverify


def run(sv, case, **kw):
    got = case.run(sv, **kw)
    check_attention(case, got)
    return got


@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (4, 4), (7, 1), (8, 1), (16, 1), (28, 4), (40, 8)])
@pytest.mark.parametrize("dim", [64, 128])
def test_heads(sv, heads, kv_heads, dim):
    run(sv, PackedAttentionCase([5, 130, 300], 1, heads, kv_heads, dim, 16))
    run(sv, PackedAttentionCase([5, 130, 300], 3, heads, kv_heads, dim, 16))


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("rows", [1, 2, 5, 40])
def test_head_dims(sv, dim, rows):
    run(sv, PackedAttentionCase([0, 1, 127, 128, 129, 400], rows, 4, 2, dim, 16, seed=dim))


@pytest.mark.parametrize("page", [1, 2, 3, 4, 5, 8, 16, 32, 64, 100, 128, 200, 256, 384])
@pytest.mark.parametrize("rows", [1, 20])
def test_pages(sv, page, rows):
    run(sv, PackedAttentionCase([3, 260, 511], rows, 8, 2, 128, page, seed=page))


@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("rows", [[1, 4, 8, 3], [17, 1, 30, 9]])
@pytest.mark.parametrize("staged", [False, True])
def test_ragged(sv, page, rows, staged):
    run(sv, PackedAttentionCase([0, 77, 300, 129], rows, 8, 2, 64, page, ragged=True, staged=staged))


@pytest.mark.parametrize("rows", [3, 17, 60])
@pytest.mark.parametrize("staged", [False, True])
def test_trees(sv, rows, staged):
    run(sv, PackedAttentionCase([0, 200, 37], rows, 4, 2, 128, 16, tree=True, staged=staged))


@pytest.mark.parametrize("lens", [[20000], [9000, 1], [1] * 90, list(range(200))])
@pytest.mark.parametrize("rows", [1, 5])
def test_lengths(sv, lens, rows):
    run(sv, PackedAttentionCase(lens, rows, 4, 1, 128, 16))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 3, 12])
def test_many_tiles_a_block(sv, dim, rows):
    """Places are used again and again, by warps that take parts of some tiles only (one request's bytes for many)."""
    case = PackedAttentionCase([6000], rows, 32, 8, dim, 16)
    cache = case.cache(sv)
    n = 24
    table = cache.page_table.expand(n, -1).contiguous()
    many = sv.PackedKvCache(cache.data, table, page_size=16, head_dim=dim)
    q = case.q.cuda().repeat(n, 1, 1)
    lens = torch.tensor([6000 - 7 * i for i in range(n)], device="cuda")
    got = sv.paged_attention(q, many, lens, max_len=rows, mask=torch.zeros(n, rows, rows, dtype=torch.uint8, device="cuda"))
    for i in (0, 5, n - 1):
        case.lens, case.mask = [6000 - 7 * i], np.zeros((1, rows, rows), np.uint8)
        one = sv.AttentionOutputs(out=got.out[i * rows:(i + 1) * rows], lse=got.lse[i * rows:(i + 1) * rows], dev_status=got.dev_status[i:i + 1])
        check_attention(case, one)
    assert (got.dev_status == 0).all()


@pytest.mark.parametrize("dim", [64, 256])
def test_long_history_of_wide_and_narrow_heads(sv, dim):
    run(sv, PackedAttentionCase([7000, 300], 1, 8, 2, dim, 16))
    run(sv, PackedAttentionCase([7000, 300], 12, 8, 2, dim, 32))


def test_head_major_blocks_and_layers(sv):
    run(sv, PackedAttentionCase([40, 300], 2, 4, 2, 128, 16, head_major=True))
    run(sv, PackedAttentionCase([40, 300], 20, 4, 2, 128, 16, head_major=True, layers=3, layer=2))


@pytest.mark.parametrize("rows", [1, 3, 24])
def test_masks_that_leave_nothing(sv, rows):
    case = PackedAttentionCase([0, 0, 200], rows, 4, 2, 64, 16, tree=True)
    case.mask[:] = 0
    got = run(sv, case)
    assert (got.out[:2 * rows] == 0).all() and torch.isneginf(got.lse[:2 * rows]).all()


@pytest.mark.parametrize("rows", [2, 24])
def test_bytes_that_no_call_writes(sv, rows):
    """New rows' entries of ones (the largest numbers) are hidden from some rows, and seen by others."""
    case = PackedAttentionCase([30, 200], rows, 4, 2, 64, 16, tree=True, q_gain=0.01)
    case.mask[:] = np.tril(np.ones((rows, rows), np.uint8))
    case.mask[:, :, 0] = 0
    case.mask[:, 0, 0] = 0
    for b in range(2):  # the first new row's entry
        x = case.lens[b]
        p, r = case.table[b, x // 16], x % 16
        parts = list(packed.unblock(case.blocks, 16, 64))
        for a in parts:
            a[0, p, r] = 255 if a.shape[-1] == 4 else 15
        case.blocks = packed.blocks(*parts)
    run(sv, case)


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0, 1e-30])
def test_scales(sv, rows, scale):
    case = PackedAttentionCase([40, 300], rows, 4, 2, 64, 16)
    case.scale = scale
    run(sv, case)


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("gain,q_gain", [(1e-5, 1.0), (3000.0, 1e-3), (1.0, 1e4), (1.0, 1e-30), (1e-3, 1e35), (100.0, 50.0)])
def test_ranges(sv, rows, gain, q_gain):
    """Scales of the cache near the ends of the format, queries beyond a half float's range."""
    case = PackedAttentionCase([40, 300], rows, 4, 2, 64, 16, gain=gain, q_gain=q_gain)
    case.scale = 1.0 / (gain * q_gain * 8.0) if gain * q_gain < 1e30 else 1e-33
    run(sv, case)


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("scale", [1e-33, 1e-37, 0.0])
def test_tiny_scales_of_a_cache_of_whole_numbers(sv, rows, scale):
    case = AttentionCase([40, 300], rows, 4, 2, 64, 16, BF16, q_gain=1e32, poison=False)
    case.scale = scale
    run(sv, case)


@pytest.mark.parametrize("rows", [1, 20])
def test_queries_of_mixed_size(sv, rows):
    case = PackedAttentionCase([40, 300], rows, 4, 2, 64, 16)
    case.q[:, 0] *= 1e20
    case.q[:, 1] *= 1e-20
    case.q[:, 2, ::2] *= 1e6
    case.q[:, 3] = 0.0
    case.scale = 1e-19
    run(sv, case)


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_queries_that_are_no_numbers(sv, rows, what):
    case = PackedAttentionCase([40, 300], rows, 4, 2, 64, 16)
    want = case.run(sv).out.clone()
    case.q[0, 1, 5] = what
    got = case.run(sv)
    assert torch.isnan(got.out[0, 1]).any() or not torch.isfinite(got.lse[0, 1])
    keep = torch.ones(case.q.shape[:2], dtype=torch.bool)
    keep[0, 1] = False
    assert torch.equal(got.out[keep.cuda()], want[keep.cuda()])


def test_bad_pages_are_reported(sv):
    for rows in (1, 20):
        case = PackedAttentionCase([40, 300, 9], rows, 4, 2, 64, 16)
        case.table[1, 3] = 10 ** 6
        case.table[2, 0] = -5
        run(sv, case)
        case = PackedAttentionCase([40, 9], rows, 4, 2, 64, 16, staged=True)
        case.row_slots[rows] = 10 ** 12
        run(sv, case)


def test_results_repeat_and_leave_the_workspace_ready(sv):
    for rows in (1, 16):
        case = PackedAttentionCase([5000, 300, 17], rows, 8, 2, 128, 16)
        ws = sv.attention_workspace(3, rows, case.cache(sv), 8)
        a = run(sv, case, ws=ws)
        for _ in range(3):
            b = case.run(sv, ws=ws)
            assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


def test_outputs_with_strides(sv):
    for rows in (1, 20):
        case = PackedAttentionCase([40, 300], rows, 4, 2, 64, 16)
        R = case.q.shape[0]
        out = sv.AttentionOutputs(out=torch.full((4, R + 1, 80), 5.0, dtype=BF16, device="cuda").transpose(0, 1)[:R, :, :64],
                                  lse=None, dev_status=torch.empty(2, dtype=torch.int32, device="cuda"))
        got = case.run(sv, out=out)
        assert torch.equal(got.out, case.run(sv).out)
