"""Attention over the paged cache against the fp64 oracle: types, head layouts, lengths around every tile edge, page
sizes, masks, staged drafts, strides, empty rows, bad pages, and the division of one request over many blocks."""
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
@pytest.mark.parametrize("lens", [[0], [1], [15, 16, 17, 31], [32, 33], [63, 64, 65], [127, 128, 129, 0, 1], [1000, 3]])
def test_decode_lengths_around_tile_edges(dtype, lens):
    check_attention(c := AttentionCase(lens, 1, 8, 2, 128, 16, dtype, seed=len(lens)), c.run(sv))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,kv,dim", [(1, 1, 8), (4, 4, 16), (8, 1, 64), (6, 2, 72), (28, 4, 80), (16, 2, 96),
                                          (40, 8, 128), (5, 1, 136), (8, 2, 256)])
def test_head_layouts(dtype, heads, kv, dim):
    check_attention(c := AttentionCase([70, 5], 3, heads, kv, dim, 16, dtype, seed=dim), c.run(sv))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [1, 3, 16, 64, 100])
@pytest.mark.parametrize("staged", [False, True])
def test_pages_and_staged_rows(dtype, page, staged):
    check_attention(c := AttentionCase([200, 77, 0], 5, 8, 4, 64, page, dtype, staged=staged, seed=page), c.run(sv))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [2, 4, 7, 16, 17, 33, 64, 100])
@pytest.mark.parametrize("tree", [False, True])
def test_new_rows_and_masks(dtype, rows, tree):
    check_attention(c := AttentionCase([90, 0, 31], rows, 8, 2, 64, 16, dtype, tree=tree, staged=tree, seed=rows), c.run(sv))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 2, 4, 7, 8, 16, 32])
def test_row_tiles_bf16(dim, group):
    # the rows of a unit (new rows times heads a cache head serves) on both sides of each tile height
    for rows in (1, 4, 5):
        c = AttentionCase([130, 64], rows, group, 1, dim, 16, BF16, seed=group)
        check_attention(c, c.run(sv))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ragged_rows(dtype):
    c = AttentionCase([5, 300, 0, 64, 1], [1, 8, 3, 5, 2], 8, 2, 128, 16, dtype, ragged=True, seed=3)
    check_attention(c, c.run(sv))
    c = AttentionCase([5, 300, 0, 64, 1], [1, 8, 3, 5, 2], 8, 2, 128, 16, dtype, ragged=True, tree=True, staged=True, seed=4)
    check_attention(c, c.run(sv))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 4, 20])
def test_one_long_request_is_split_and_joined(dtype, rows):
    c = AttentionCase([20011], rows, 4, 1, 64, 32, dtype, seed=9)
    check_attention(c, c.run(sv))


def test_many_requests():
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 60, 700).tolist()
    check_attention(c := AttentionCase(lens, 1, 2, 1, 64, 16, BF16, seed=5), c.run(sv))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_head_major_pages_and_layers(dtype):
    c = AttentionCase([100, 33], 4, 8, 4, 64, 16, dtype, head_major=True, layers=3, layer=2, seed=11)
    check_attention(c, c.run(sv))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_q_and_out(dtype):
    c = AttentionCase([100, 33], 3, 8, 4, 64, 16, dtype, seed=12)
    big = torch.randn(6, 8 + 4 + 4, 64).to(dtype).cuda()  # q inside a fused projection
    big[:, :8] = c.q.cuda()
    c.q = big[:, :8].cpu()
    obuf = torch.full((6, 2, 8, 64), 7.0, dtype=dtype, device="cuda")
    out = sv.AttentionOutputs.allocate(6, 8, 64, 2, dtype)
    out.out = obuf[:, 1]
    cache_q = big[:, :8]
    real, c.q = c.q, cache_q
    got = c.run(sv, out=out)
    c.q = real
    check_attention(c, got)
    assert (obuf[:, 0] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_that_see_nothing(dtype):
    c = AttentionCase([0, 40, 0], 6, 4, 2, 64, 16, dtype, tree=True, staged=True, seed=13)
    c.mask[0, 2] = 0      # no history and no visible row
    c.mask[2] = 0
    got = c.run(sv)
    check_attention(c, got)
    assert (got.out[2] == 0).all() and torch.isneginf(got.lse[2]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("group", [1, 8])
def test_unseen_rows_do_not_leak(dtype, bad, group):
    # node 2's K/V hold what must not reach the rows that do not see it
    for rows in (5, 13):
        c = AttentionCase([37], rows, 2 * group, 2, 128, 16, dtype, tree=True, staged=True, seed=14)
        c.mask[0, :, 2] = 0
        c.mask[0, 2, 2] = 1
        s = int(c.row_slots[2])
        c.k[0, s // 16, s % 16] = bad
        c.v[0, s // 16, s % 16, :, ::3] = bad
        got, o = c.run(sv), c.oracle()
        others = [i for i in range(rows) if i != 2]
        assert torch.isfinite(got.out[others]).all()
        ref = torch.from_numpy(o["out"][others])
        assert (got.out[others].double().cpu() - ref).abs().max() < 0.05
        # the row that sees it follows its formula: NaN where the exact result is NaN
        if bad != bad:
            assert torch.isnan(got.out[2]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scores_far_apart(dtype):
    c = AttentionCase([300], 3, 4, 2, 64, 16, dtype, seed=15, q_gain=200.0)
    check_attention(c, c.run(sv))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bad_pages_slots_and_lengths_are_reported(dtype):
    c = AttentionCase([100, 50, 20, 33], 2, 4, 2, 64, 16, dtype, staged=True, seed=16)
    c.table[0, 3] = 10 ** 6
    c.table[1, 1] = -1
    c.row_slots[5] = -3
    c.row_slots[6] = 1 << 40
    got = c.run(sv)
    check_attention(c, got)
    assert got.dev_status.tolist() == [128, 128, 128, 128]
    c = AttentionCase([100, 50], 2, 4, 2, 64, 16, dtype, seed=17)
    c.lens = [-5, 100000]
    check_attention(c, c.run(sv))


def test_bad_row_ranges_leave_their_rows():
    c = AttentionCase([10, 20, 30], [2, 3, 1], 4, 2, 64, 16, BF16, ragged=True, seed=18)
    good = c.run(sv)
    c.cu = np.array([0, 2, 2, 6], np.int32)  # an empty request, then one longer than max_len
    out = sv.AttentionOutputs.allocate(6, 4, 64, 3, BF16)
    out.out.fill_(3.0)
    got = c.run(sv, out=out)
    assert got.dev_status.tolist() == [0, 8, 8]
    assert torch.equal(got.out[:2], good.out[:2]) and (got.out[2:] == 3.0).all()


def test_repeats_are_bit_equal_and_the_workspace_rewinds():
    c = AttentionCase([5000, 3, 900], 5, 8, 2, 128, 16, BF16, seed=19)
    first = c.run(sv)
    ws = torch.zeros_like(sv.attention_workspace(3, 5, sv.PagedKvCache(c.dk, c.dv, c.dtable), 8))
    for _ in range(3):
        again = c.run(sv, ws=ws)
        assert torch.equal(first.out, again.out) and torch.equal(first.lse, again.lse)
    d = AttentionCase([70], 1, 2, 2, 128, 16, BF16, seed=20)
    check_attention(d, d.run(sv, ws=ws))  # another shape on the same workspace
    assert torch.equal(first.out, c.run(sv, ws=ws).out)


@pytest.mark.parametrize("rows,dim", [(17, 64), (33, 128), (64, 64), (64, 128)])
def test_many_rows_repeat_bit_equal_with_short_segments(rows, dim):
    # about two key tiles a block: the end of a unit follows its beginning at once
    c = AttentionCase([20011], rows, 4, 1, dim, 32, BF16, seed=9)
    first = c.run(sv)
    check_attention(c, first)
    for _ in range(12):
        again = c.run(sv)
        assert torch.equal(first.out, again.out) and torch.equal(first.lse, again.lse)


def test_side_stream():
    c = AttentionCase([900, 70], 2, 8, 2, 128, 16, BF16, seed=21)
    ref = c.run(sv)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(sv, stream=s)
    s.synchronize()
    assert torch.equal(ref.out, got.out)


def test_offsets_past_32_bits():
    # 5 GB of cache: pages whose byte offsets pass 2^32, reached through the table
    pages, page, G, D = 80000, 16, 8, 128
    k = torch.zeros(1, pages, page, G, D, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(3)
    use = torch.tensor([79999, 70001, 5, 66000], device="cuda")
    k[0, use] = torch.randn(4, page, G, D, generator=g, device="cuda").to(BF16)
    v[0, use] = torch.randn(4, page, G, D, generator=g, device="cuda").to(BF16)
    q = torch.randn(1, 16, D, generator=g, device="cuda").to(BF16)
    L = torch.tensor([60], device="cuda")
    big = sv.paged_attention(q, sv.PagedKvCache(k, v, use.int()[None]), L)
    small = sv.paged_attention(q, sv.PagedKvCache(k[:, use].clone(), v[:, use].clone(),
                                                  torch.arange(4, dtype=torch.int32, device="cuda")[None]), L)
    assert torch.equal(big.out, small.out) and big.dev_status.tolist() == [0]
