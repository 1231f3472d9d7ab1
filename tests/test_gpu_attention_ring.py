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
from tests.serving_cases import BF16, F32, AttentionCase, attention_bounds, check_attention  # noqa: E402


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


def check_rows(case, got, keep, exact_scores=False):
    """check_attention for the rows `keep` alone; exact_scores: fp32 holds all of their scores' sums exactly."""
    o = case.oracle()
    if exact_scores:
        o["smax"][:] = 0.0
    tol, lse_tol = attention_bounds(o, case.q.shape[2], case.dtype)
    out, lse = got.out.double().cpu().numpy(), got.lse.double().cpu().numpy()
    assert np.isfinite(out[keep]).all()
    assert (np.abs(out - o["out"])[keep] <= tol[keep]).all()
    assert np.array_equal(np.isneginf(lse[keep]), np.isneginf(o["lse"][keep]))
    fine = np.isfinite(o["lse"][keep])
    assert (np.abs(lse[keep][fine] - o["lse"][keep][fine]) <= lse_tol[keep][fine]).all()
    assert np.array_equal(got.dev_status.cpu().numpy().view(np.uint32), o["status"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 136, 256])
@pytest.mark.parametrize("rows", [4, 20])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_of_unseen_rows_behind_long_histories(dtype, dim, rows, bad):
    # every request's third row holds what only it sees, behind histories of several tiles
    c = AttentionCase([900, 260, 37, 128, 511, 0, 1300], rows, 8, 2, dim, 16, dtype, tree=True, staged=True, seed=dim + rows)
    R = rows * len(c.lens)
    for b in range(len(c.lens)):
        c.mask[b, :, 2] = 0
        c.mask[b, 2, 2] = 1
        s = int(c.row_slots[b * rows + 2])
        c.k[0, s // 16, s % 16] = bad
        c.v[0, s // 16, s % 16, :, ::3] = bad
    got = c.run(sv)
    check_rows(c, got, [r for r in range(R) if r % rows != 2])
    for _ in range(3):
        again = c.run(sv)
        assert torch.equal(torch.nan_to_num(got.out), torch.nan_to_num(again.out))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [2, 8])
def test_every_other_row_holds_no_number(dtype, dim, heads):
    # a lane takes the values out that other lanes of its warp read next
    for rows in (4, 8):
        c = AttentionCase([120, 0, 640, 57] * 4, rows, heads, 2, dim, 16, dtype, tree=True, staged=True, seed=dim + rows)
        c.mask[:] = 0
        c.mask[:, ::2, ::2] = np.tril(np.ones((rows // 2, rows // 2), np.uint8))
        for s in c.row_slots.reshape(-1, rows)[:, 1::2].ravel():
            c.k[0, s // 16, s % 16], c.v[0, s // 16, s % 16] = float("nan"), float("-inf")
        first = c.run(sv)
        check_rows(c, first, list(range(len(c.q))))
        for _ in range(5):
            assert torch.equal(first.out, c.run(sv).out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads", [4, 40])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_single_row_that_does_not_see_itself(dtype, heads, bad):
    for ragged in (False, True):
        c = AttentionCase([300, 0, 37, 128], [1, 2, 1, 1] if ragged else 1, heads, 2, 128, 16, dtype, tree=True, staged=True,
                          ragged=ragged, seed=heads)
        c.mask[:] = 0
        for s in c.row_slots:
            c.k[0, s // 16, s % 16] = bad
            c.v[0, s // 16, s % 16, :, ::3] = bad
        check_rows(c, c.run(sv), list(range(len(c.q))))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 20])
def test_an_output_of_heads_before_rows(dtype, rows):
    c = AttentionCase([300, 37], rows, 8, 2, 64, 16, dtype, seed=rows)
    out = sv.AttentionOutputs.allocate(2 * rows, 8, 64, 2, dtype)
    out.out = torch.empty(8, 2 * rows, 64, dtype=dtype, device="cuda").transpose(0, 1)
    check_attention(c, c.run(sv, out=out))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 3, 18])
@pytest.mark.parametrize("power", [10, 24, 31, 40, 80, 120])
def test_largest_scores(dtype, rows, power):
    # scores of a whole number times 2^power: the weights are 0, or shared by the keys that have the largest one
    c = AttentionCase([300, 37, 0, 1300], rows, 8, 2, 64, 16, dtype, seed=power + rows, poison=False)
    g = torch.Generator().manual_seed(power)
    c.q = torch.zeros_like(c.q)
    c.q[..., 5] = 2.0 ** power * (1 - 2 * torch.randint(0, 2, c.q.shape[:2], generator=g)).to(dtype)
    c.k[..., 5] = torch.randint(-40, 41, c.k.shape[:-1], generator=g).to(dtype)
    for c.scale in (1.0, -2.0):
        check_rows(c, c.run(sv), list(range(len(c.q))), exact_scores=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 3, 18])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_only_scores_of_minus_infinity_give_zero(dtype, rows, bad):
    # no history; every new row sees new row 0 (and the last one itself), whose scores are -inf and whose V holds no number
    c = AttentionCase([0, 0], rows, 8, 2, 64, 16, dtype, tree=True, staged=True, seed=rows)
    c.q[..., 5] = 1.0
    c.mask[:] = 0
    c.mask[:, :, 0] = 1
    c.mask[:, rows - 1, rows - 1] = 1
    for s in c.row_slots.reshape(2, rows)[:, 0]:
        c.k[0, s // 16, s % 16] = 0.0
        c.k[0, s // 16, s % 16, :, 5] = -float("inf")
        c.v[0, s // 16, s % 16, :, ::3] = bad
    got = c.run(sv)
    for b in range(2):
        for i in range(rows - 1 if rows > 1 else 1):
            assert torch.isneginf(got.lse[b * rows + i]).all() and (got.out[b * rows + i] == 0).all(), (b, i)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 4])
def test_weights_of_few_rows_keep_more_than_eight_bits(dim, rows):
    # outputs near 0, sums of terms that cancel: weights rounded once, by 2^-9, would miss them by far more than their own
    # last place
    c = AttentionCase([5, 300, 1100], rows, 4, 1, dim, 16, BF16, seed=dim + rows)
    o = c.oracle()
    got = c.run(sv).out.double().cpu().numpy()
    # an fp32 computation's bound, the rounding of what a weight's upper half leaves (2^-9 of 2^-7), and the result's one
    fp32, _ = attention_bounds(o, dim, F32)
    tol = fp32 + 2.0 ** -16 * o["mag"] + 2.0 ** -8 * np.abs(o["out"])
    assert (np.abs(got - o["out"]) <= tol).all(), float((np.abs(got - o["out"]) / tol).max())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 3, 18])
def test_infinities_in_the_history_stay_infinities(dtype, rows):
    # a weight above 0 times an infinity, and finite terms beside it; scores close together, so that no weight vanishes
    c = AttentionCase([300, 37, 700], rows, 8, 2, 64, 16, dtype, seed=rows, q_gain=0.5)
    for b in range(3):
        for x, sign in ((0, 1.0), (20, 1.0), (36, -1.0)):
            page = int(c.table[b, x // 16])
            c.v[0, page, x % 16, :, 7 if sign > 0 else 9] = sign * float("inf")
    got, o = c.run(sv), c.oracle()
    out = got.out.double().cpu().numpy()
    assert np.isposinf(o["out"][:, :, 7]).all() and np.isneginf(o["out"][:, :, 9]).all()
    assert np.isposinf(out[:, :, 7]).all() and np.isneginf(out[:, :, 9]).all()
    finite = [d for d in range(64) if d not in (7, 9)]
    tol, _ = attention_bounds(o, 64, dtype)
    assert (np.abs(out[:, :, finite] - o["out"][:, :, finite]) <= tol[:, :, finite]).all()
