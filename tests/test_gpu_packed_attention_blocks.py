"""Attention over the 4-bit cache of blocks of many rows: several tiles of 128 rows a unit's request, and units of more than 64 rows
in long lines of tiles."""
import numpy as np
import pytest
import torch

from tests.packed_cases import PackedAttentionCase
from tests.serving_cases import check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    from reject_row_vocab_gb300 import specverify
    return specverify


def run_twice(sv, case):
    first, again = case.run(sv), case.run(sv)
    check_attention(case, first)
    assert torch.equal(first.out, again.out) and torch.equal(first.lse, again.lse)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [127, 129, 257, 1024])
@pytest.mark.parametrize("history", [0, 700])
def test_causal_blocks(sv, dim, rows, history):
    run_twice(sv, PackedAttentionCase([history], rows, 2, 1, dim, 16, seed=rows + history))


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("page", [1, 16, 48, 128])
@pytest.mark.parametrize("staged", [False, True])
def test_causal_blocks_of_several_requests(sv, dim, page, staged):
    run_twice(sv, PackedAttentionCase([130, 0, 64, 1], [200, 300, 129, 1], 4, 2, dim, page, ragged=True, staged=staged, seed=dim))


@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("rows", [2, 3, 20, 130])
@pytest.mark.parametrize("shape", ["all", "upper", "random", "none"])
def test_masks_of_any_shape(sv, dim, rows, shape):
    case = PackedAttentionCase([200, 0, 128], rows, 8, 2, dim, 16, tree=True, staged=True, seed=rows)
    full = np.ones((3, rows, rows), np.uint8)
    case.mask = {"all": full, "upper": np.triu(full), "none": 0 * full,
                 "random": (np.random.default_rng(rows).random(full.shape) < 0.4).astype(np.uint8) * 255}[shape]
    check_attention(case, case.run(sv))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("rows", [[20], [40, 40, 23, 40, 33]])
def test_many_tiles_a_block(sv, dim, page, rows):
    """80 to 160 rows a unit over 2900 keys, each tile's places used again and again: trees whose rows cross the end of a row tile, and
    a last row tile that is not full.  (One request's bytes and tree for all of them.)"""
    most, heads, G, n = max(rows), 16, 4, 30
    case = PackedAttentionCase([2900], most, heads, G, dim, page, tree=True, staged=True, seed=most)
    cache, o = case.cache(sv), case.oracle()
    many = sv.PackedKvCache(cache.data, cache.page_table.expand(n, -1).contiguous(), page_size=page, head_dim=dim)
    count = [rows[b % len(rows)] for b in range(n)]
    pick = torch.cat([torch.arange(c) for c in count])
    q, slots = case.q[pick].cuda(), torch.from_numpy(case.row_slots)[pick].cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(count)]), dtype=torch.int32, device="cuda")
    got = sv.paged_attention(q, many, torch.full((n,), 2900, device="cuda"), max_len=most, cu_seqlens=cu, row_slots=slots,
                             mask=torch.from_numpy(case.mask).cuda().expand(n, -1, -1).contiguous(), scale=case.scale)
    assert (got.dev_status == 0).all()
    at = 0
    for c in count:  # (a request's first rows see no later ones: their results are those of the whole tree)
        case.q = q[at:at + c]
        case.oracle = lambda c=c: {**{k: v[:c] for k, v in o.items() if k != "status"}, "status": o["status"]}
        check_attention(case, sv.AttentionOutputs(out=got.out[at:at + c], lse=got.lse[at:at + c], dev_status=got.dev_status[:1]))
        at += c
