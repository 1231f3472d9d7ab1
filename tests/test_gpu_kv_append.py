"""Rows appended to a KV cache, and read back, against the fp64 oracle: types, layouts, positions, places, refusals on the
device."""
import numpy as np
import pytest
import torch

from oracle import packed
from tests.packed_cases import AppendCase, check_append
from tests.serving_cases import BF16, F32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    from reject_row_vocab_gb300 import specverify
    return specverify


def run(sv, case, **kw):
    d = case.make(sv)
    got = case.append(sv, d, **kw)
    check_append(case, d, got)
    return d, got


BOTH = pytest.mark.parametrize("is_packed", [False, True])


@BOTH
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,pairs,interleaved", [
    (128, None, False), (128, None, True), (64, 16, False), (64, 16, True), (96, 24, False), (128, 5, False), (128, 37, False),
    (256, None, False), (256, 128, True), (32, 1, True), (32, 16, False), (160, 80, False), (128, 0, False)])
def test_dims_and_pairs(sv, is_packed, dtype, dim, pairs, interleaved):
    run(sv, AppendCase([7, 0, 33], 3, 4, 2, dim, 16, dtype, is_packed=is_packed, pairs=pairs, interleaved=interleaved, seed=dim))


@pytest.mark.parametrize("dtype,dim,pairs", [(BF16, 8, 4), (BF16, 80, 40), (BF16, 24, 9), (F32, 4, 2), (F32, 12, 6), (F32, 100, 50)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_narrow_and_odd_heads(sv, dtype, dim, pairs, interleaved):
    run(sv, AppendCase([3, 20], 2, 3, 3, dim, 8, dtype, pairs=pairs, interleaved=interleaved))


@BOTH
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (7, 1), (28, 4), (12, 12), (64, 8)])
def test_heads(sv, is_packed, heads, kv_heads):
    run(sv, AppendCase([5, 9], [1, 4], heads, kv_heads, 64, 16, BF16, is_packed=is_packed, ragged=True))


@BOTH
@pytest.mark.parametrize("page", [1, 2, 5, 16, 64, 200])
@pytest.mark.parametrize("staged", [False, True])
def test_pages_and_places(sv, is_packed, page, staged):
    run(sv, AppendCase([0, 1, 31, 100], [3, 1, 8, 20], 8, 2, 128, page, BF16, is_packed=is_packed, ragged=True, staged=staged))


@BOTH
@pytest.mark.parametrize("lens,rows", [([0], 1), ([511], 1), ([3] * 300, 1), ([0, 700], [900, 1]), ([5] * 70, [0, 1] * 35),
                                       ([10, 20, 30], [0, 0, 5]), ([1] * 2100, [1, 0, 2] * 700)])
def test_lengths(sv, is_packed, lens, rows):
    run(sv, AppendCase(lens, rows, 4, 2, 64, 16, BF16, is_packed=is_packed, ragged=not isinstance(rows, int), spare_rows=3))


@BOTH
def test_given_positions(sv, is_packed):
    far = [0, 1, 5, 1_000_003, 2 ** 24 + 1, 2 ** 30 + 7, 4, 4]
    run(sv, AppendCase([2, 9], 4, 4, 2, 64, 16, F32, is_packed=is_packed, positions=far, magnitude=1.25))


def test_angles_of_far_positions(sv):
    """A rotation by the position alone: cosines and sines of angles up to 2^31, to fp32."""
    pos = np.array([0, 1, 12345, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 1], np.int64)
    case = AppendCase([0] * 6, 1, 1, 1, 64, 16, F32, positions=pos)
    case.qkv[:, 0, :32], case.qkv[:, 0, 32:] = 1.0, 0.0
    d = case.make(sv)
    out = case.append(sv, d).q.double().cpu().numpy()[:, 0]
    angle = pos[:, None].astype(np.float64) * case.inv_freq.astype(np.float64)
    assert np.abs(out[:, :32] - np.cos(angle)).max() <= 3 * 2.0 ** -23
    assert np.abs(out[:, 32:] - np.sin(angle)).max() <= 3 * 2.0 ** -23


@BOTH
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_farthest_positions(sv, is_packed, dtype):
    """Positions of 2^31 and beyond, to the ends of 64 bits."""
    rng = np.random.default_rng(3)
    pos = np.array([2 ** 31 + 5, -(2 ** 33) - 1, 2 ** 40 + 12345, 2 ** 52 + 3, 2 ** 53 + 1, -(2 ** 60) + 11, 2 ** 63 - 1, -(2 ** 63)] +
                   [int(x) for x in rng.integers(2 ** 31, 2 ** 62, 24)], np.int64)
    run(sv, AppendCase([0] * 32, 1, 4, 2, 64, 16, dtype, is_packed=is_packed, positions=pos))


@BOTH
def test_without_rotation_and_without_queries(sv, is_packed):
    case = AppendCase([7, 3], 2, 2, 2, 64, 16, BF16, is_packed=is_packed, rotation=False)
    d = case.make(sv)
    check_append(case, d, case.append(sv, d, q=False), q=False)
    d = case.make(sv)
    got = case.append(sv, d)
    check_append(case, d, got)
    assert torch.equal(got.q, d["qkv"][:, :2])


@BOTH
@pytest.mark.parametrize("pairs", [32, 13])
def test_queries_in_place(sv, is_packed, pairs):
    case = AppendCase([7, 3, 90], 5, 16, 2, 64, 16, BF16, is_packed=is_packed, pairs=pairs)
    d = case.make(sv)
    want = case.append(sv, case.make(sv)).q
    qkv = d["qkv"].clone()
    out = sv.KvAppendOutputs(q=d["qkv"][:, :16], dev_status=torch.zeros(3, dtype=torch.int32, device="cuda"))
    check_append(case, d, case.append(sv, d, out=out))
    assert torch.equal(d["qkv"][:, :16], want) and torch.equal(d["qkv"][:, 16:], qkv[:, 16:])


@BOTH
def test_one_layer_of_several(sv, is_packed):
    run(sv, AppendCase([7, 3], 2, 2, 2, 64, 16, BF16, is_packed=is_packed, layers=3, layer=2))


def test_head_major_cache_and_queries(sv):
    case = AppendCase([7, 30], 3, 4, 2, 64, 16, BF16)
    d = case.make(sv)
    major = [d[n].transpose(2, 3).contiguous().transpose(2, 3) for n in ("k", "v")]
    d["k"], d["v"] = major
    d["cache"] = sv.PagedKvCache(*major, d["table"])
    out = sv.KvAppendOutputs(q=torch.empty(4, 6, 64, dtype=BF16, device="cuda").transpose(0, 1),
                             dev_status=torch.zeros(2, dtype=torch.int32, device="cuda"))
    check_append(case, d, case.append(sv, d, out=out))


@BOTH
def test_rows_of_no_request_are_left(sv, is_packed):
    case = AppendCase([7, 3], [2, 1], 4, 2, 64, 16, BF16, is_packed=is_packed, ragged=True, spare_rows=4)
    d = case.make(sv)
    out = sv.KvAppendOutputs.allocate(case.total, 4, 64, 2)
    out.q.fill_(7.0)
    check_append(case, d, case.append(sv, d, out=out))
    assert (out.q[3:] == 7.0).all()
    back = sv.KvReadOutputs.allocate(case.total, 2, 64, 2)
    back.k.fill_(7.0), back.v.fill_(7.0)
    case.read(sv, d, out=back)
    assert (back.k[3:] == 7.0).all() and (back.v[3:] == 7.0).all()


@BOTH
def test_bad_places_and_ranges_are_reported(sv, is_packed):
    case = AppendCase([7, 3, 40, 2], 2, 2, 2, 64, 4, BF16, is_packed=is_packed)
    case.table[2, 10] = 10 ** 6  # positions 40 and 41
    case.lens[3] = -1
    run(sv, case)
    case = AppendCase([7, 3], 3, 2, 2, 64, 4, BF16, is_packed=is_packed, staged=True)
    case.row_slots[1], case.row_slots[4] = -1, case.pages * 4
    run(sv, case)
    case = AppendCase([7, 3, 5, 6], [3, 2, 2, 1], 2, 2, 64, 4, BF16, is_packed=is_packed, ragged=True)
    case.max_len = 2  # the first request has too many rows
    run(sv, case)
    case = AppendCase([7, 3, 5], [2, 2, 2], 2, 2, 64, 4, BF16, is_packed=is_packed, ragged=True)
    case.cu = np.array([0, 2, 100, 6], np.int32)  # past the rows, and decreasing
    run(sv, case)
    case.cu = np.array([4, 6, 1, 3], np.int32)  # the second decreases; the others' rows are stored
    run(sv, case)


@BOTH
def test_past_the_page_table(sv, is_packed):
    case = AppendCase([14, 3], 2, 2, 2, 64, 4, BF16, is_packed=is_packed)
    case.lens[0] = case.table.shape[1] * 4 - 1  # its second row is past the table
    run(sv, case)
    case.lens[0] = 2 ** 40
    case.positions = np.arange(4)
    run(sv, case)


def test_numbers_at_the_ends_of_the_format(sv):
    """Values copied without rotation: groups of zeros, of the smallest and the largest numbers, ties, infinities and NaN."""
    case = AppendCase([3, 9], 16, 1, 1, 64, 16, F32, is_packed=True, rotation=False)
    x = case.qkv[:, 1:]
    for r in range(16):
        x[r] *= 2.0 ** (r * 4 - 40)          # scales from below the smallest to the largest
    x[16] = 0.0
    x[17, :, ::2] = -0.0
    codes = torch.from_numpy(packed.MAGNITUDES).float()
    x[18, :, :8], x[18, :, 8:16] = codes, -codes                       # codes as they are
    mid = (codes[1:] + codes[:-1]) / 2
    x[19, :, :7], x[19, :, 7] = mid * 0.75, 6.0 * 0.75                 # half way between two codes
    x[20, :, :7], x[20, :, 7] = torch.nextafter(mid, torch.tensor(9.0)) * 1.0, 6.0
    x[21, :, :7], x[21, :, 7] = torch.nextafter(mid, torch.tensor(0.0)) * 1.0, 6.0
    s = torch.from_numpy(packed.SCALES).float()
    for k in range(4):
        half = (s[60 + k] + s[61 + k]) / 2
        x[22, 0, 16 * k:16 * k + 16] = 6.0 * half                      # half way between two scales
        x[23, 0, 16 * k:16 * k + 16] = torch.nextafter(6.0 * half, torch.tensor(0.0))
        x[24, 0, 16 * k:16 * k + 16] = 6.0 * s[60 + k]
    x[25, 0, 3], x[25, 1, 40] = float("inf"), float("-inf")
    x[26, 0, 5] = float("nan")
    x[27, 0] = 3e38
    x[28, 0, :16] = 1e-45
    run(sv, case)


def test_every_scale_and_tie_of_bf16(sv):
    """All multiples that bf16 has of a scale, against the oracle's search."""
    case = AppendCase([0], 512, 1, 1, 128, 16, BF16, is_packed=True, rotation=False)
    g = torch.Generator().manual_seed(5)
    scale = torch.from_numpy(packed.SCALES).float()[torch.randint(1, packed.MOST + 1, (512, 2, 8, 1), generator=g)]
    steps = torch.randint(-48, 49, (512, 2, 8, 16), generator=g) / 8.0
    case.qkv[:, 1:] = (scale * steps).reshape(512, 2, 128).to(BF16)
    run(sv, case)


@pytest.mark.parametrize("dtype,pairs,interleaved,magnitude", [(BF16, 64, False, 1.0), (BF16, 64, True, 1.25), (F32, 64, False, 1.0),
                                                               (F32, 19, True, 1.0), (BF16, 29, False, 0.75)])
def test_keys_are_stored_as_exact_rotations_would_be(sv, dtype, pairs, interleaved, magnitude):
    """Every scale and code of a million rotated keys, those among them that a rotation in fp32 puts on a border's other side.  (64-bit
    angles are off by 2^-40 here: a key that close to a border is one in 10^10.)"""
    case = AppendCase([0, 3000, 100000], 700, 1, 4, 128, 16, dtype, is_packed=True, staged=True, pairs=pairs, interleaved=interleaved,
                      magnitude=magnitude, seed=pairs)
    d = case.make(sv)
    got = case.append(sv, d)
    o = case.oracle()
    assert (got.dev_status == 0).all() and (o["slot"] >= 0).all()
    parts = packed.unblock(d["data"].cpu().numpy(), 16, 128)
    codes, scales = (t[0].reshape(-1, 4, t.shape[-1])[o["slot"]] for t in parts[:2])
    _, want_scales, want = packed.quantize(o["k"])
    assert np.array_equal(scales, want_scales)
    assert np.array_equal(packed.values(codes, scales), want)


@pytest.mark.parametrize("dim,pairs,interleaved", [(32, 8, True), (64, 16, False), (64, 13, False)])
@pytest.mark.parametrize("start", [100, 4000, 20_000, 100_000, 10 ** 6, 2 ** 22 - 64, 2 ** 22, 2 ** 30 + 1, 2 ** 44 + 3])
def test_keys_next_to_a_border(sv, dim, pairs, interleaved, start):
    """Values that lie 2^-34 to 2^-33 beside the middle of two codes, at near and far positions.  (What may be off by rounding: sines
    and cosines by 2^-37 each, of pairs of up to 4 together.)"""
    rng = np.random.default_rng(pairs + start)
    case = AppendCase([0] * 64, 1, 1, 1, dim, 16, F32, is_packed=True, staged=True, pairs=pairs, interleaved=interleaved,
                      positions=start + np.arange(64))
    case.inv_freq = rng.uniform(0.3, 1.0, pairs).astype(np.float32)
    case.inv_freq[-1] = 0.0  # a pair that nothing turns, (6, 0), gives the group of columns 0 .. 15 its scale of 1
    first, second = (np.arange(pairs) * 2, np.arange(pairs) * 2 + 1) if interleaved else (np.arange(pairs), np.arange(pairs) + pairs)
    angle = packed.angles(case.positions, case.inv_freq)
    key, planted = case.qkv[:, 1].numpy(), np.zeros((64, pairs), bool)
    key[:, first[-1]], key[:, second[-1]] = 6.0, 0.0
    for r in range(64):
        for i in range(pairs - 1):
            c, s, border = np.cos(angle[r, i]), np.sin(angle[r, i]), rng.choice([0.25, 0.75, 1.25])
            x = rng.uniform(0.5, 1.5, 4000).astype(np.float32).astype(np.float64)
            y = ((x * c - border) / s).astype(np.float32).astype(np.float64) if abs(s) > 0.1 else x
            off = np.abs((x * c - border) - y * s)
            good = np.nonzero((off >= 2.0 ** -34) & (off <= 2.0 ** -33) & (np.abs(x) + np.abs(y) <= 4.0))[0]
            j = good[0] if len(good) else 0
            planted[r, i] = len(good) > 0
            key[r, first[i]], key[r, second[i]] = x[j], y[j] if len(good) else 0.0
    assert planted.mean() > 0.5
    d = case.make(sv)
    assert (case.append(sv, d).dev_status == 0).all()
    o = case.oracle()
    assert (np.abs(np.abs(o["k"][:, 0, first][planted][:, None] - [0.25, 0.75, 1.25]).min(1) - 1.5 * 2.0 ** -34) <= 2.0 ** -34).all()
    parts = packed.unblock(d["data"].cpu().numpy(), 16, dim)
    codes, scales = (t[0].reshape(-1, 1, t.shape[-1])[o["slot"]] for t in parts[:2])
    want_codes, want_scales, want = packed.quantize(o["k"])
    assert np.array_equal(scales, want_scales) and (packed.SCALES[scales[:, 0, 0]] == 1.0).all()
    assert np.array_equal(packed.values(codes, scales), want)


@BOTH
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,page,staged", [(64, 16, False), (128, 1, True), (256, 5, False), (96, 16, True)])
def test_read_back(sv, is_packed, dtype, dim, page, staged):
    case = AppendCase([7, 0, 50], [1, 6, 30], 2, 2, dim, page, dtype, is_packed=is_packed, ragged=True, staged=staged, layers=2,
                      layer=1)
    d = case.make(sv)
    got = case.append(sv, d)
    check_append(case, d, got)
    o = case.oracle()
    r = case.read(sv, d, layer=1)
    every = case.read(sv, d, layer=None)
    assert torch.equal(every.k[1], r.k) and torch.equal(every.v[1], r.v) and (r.dev_status == 0).all()
    assert not torch.equal(every.k[0], r.k)
    if is_packed:
        parts = packed.unblock(d["data"].cpu().numpy(), page, dim)
        want = [packed.values(parts[i], parts[i + 1])[1].reshape(-1, 2, dim)[o["slot"]] for i in (0, 2)]
    else:
        want = [d[n][1].double().cpu().numpy().reshape(-1, 2, dim)[o["slot"]] for n in ("k", "v")]
    for have, w in zip((r.k, r.v), want):
        assert np.array_equal(have.double().cpu().numpy(), w)


@BOTH
def test_read_of_bad_places_is_zero(sv, is_packed):
    case = AppendCase([7, 3], 3, 2, 2, 64, 4, BF16, is_packed=is_packed, staged=True)
    d = case.make(sv)
    case.append(sv, d)
    d["slots"][1], d["slots"][5] = -3, 10 ** 12
    r = case.read(sv, d)
    assert (r.k[[1, 5]] == 0).all() and (r.v[[1, 5]] == 0).all() and (r.k[[0, 2]] != 0).any()
    assert r.dev_status.tolist() == [128, 128]


def test_status_collects_over_calls(sv):
    case = AppendCase([7, 3], 1, 2, 2, 64, 4, BF16, is_packed=True)
    d = case.make(sv)
    out = sv.KvAppendOutputs.allocate(2, 2, 64, 2)
    d["qkv"][1, 2, 0] = float("inf")
    case.append(sv, d, out=out)
    d["qkv"][1, 2, 0] = 1.0
    d["table"][0] = -1
    case.append(sv, d, out=out)
    assert out.dev_status.tolist() == [128, 2]


@BOTH
def test_large_offsets(sv, is_packed):
    """A cache of more than 2^32 bytes, places at its end."""
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB")
    page, heads, dim = 64, 8, 128
    pages = (9 << 30) // (page * heads * dim * (2 if not is_packed else 1) * 9 // 8) if is_packed else (5 << 30) // (page * heads * dim * 2)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    if is_packed:
        cache = sv.PackedKvCache.allocate(1, pages, heads, page, dim, table)
        assert cache.data.numel() > 1 << 32
    else:
        cache = sv.PagedKvCache(*(torch.zeros(1, pages, page, heads, dim, dtype=BF16, device="cuda") for _ in range(2)), table)
        assert cache.k.numel() * 2 > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(70, heads, dim, generator=g, device="cuda").to(BF16) for _ in range(2))
    start = torch.zeros(1, dtype=torch.int64, device="cuda")
    sv.kv_append(cache, k, v, seq_lens=start, max_len=70)
    r = sv.kv_read(cache, layer=0, seq_lens=start, max_len=70)
    want = (k, v) if not is_packed else [torch.from_numpy(packed.quantize(t.double().cpu().numpy())[2]).to(BF16).cuda() for t in (k, v)]
    assert torch.equal(r.k, want[0]) and torch.equal(r.v, want[1]) and r.dev_status.item() == 0
