"""Attention over the 4-bit cache against the fp64 oracle on the values that the cache stands for."""
import numpy as np
import pytest
import torch

from oracle import packed
from tests.packed_cases import PackedAttentionCase
from tests.serving_cases import BF16, AttentionCase, attention_bounds, check_attention

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


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 3, 12, 40])
def test_many_units_a_block(sv, dim, rows):
    """Units of one tile or two in quick turn, a dozen a block or more: the plan's places are used again, and each unit's queries are
    those of its own request and head.  (One request's bytes for all; the new rows are hidden.)"""
    n, heads, G = 500, 8, 4
    case = PackedAttentionCase([200], rows, heads, G, dim, 16)
    cache = case.cache(sv)
    many = sv.PackedKvCache(cache.data, cache.page_table.expand(n, -1).contiguous(), page_size=16, head_dim=dim)
    g = torch.Generator(device="cuda").manual_seed(rows)
    q = (2.0 * torch.randn(n * rows, heads, dim, device="cuda", generator=g)).to(BF16)
    lens = torch.tensor([1 + 37 * b % 200 for b in range(n)], device="cuda")
    call = lambda: sv.paged_attention(q, many, lens, max_len=rows, scale=case.scale,
                                      mask=torch.zeros(n, rows, rows, dtype=torch.uint8, device="cuda"))
    got, again = call(), call()
    assert torch.equal(got.out, again.out) and torch.equal(got.lse, again.lse) and (got.dev_status == 0).all()
    x = torch.arange(200)
    slot = torch.from_numpy(case.table[0])[x // 16].long() * 16 + x % 16
    k, v = (t[0].reshape(-1, G, dim)[slot].cuda().repeat_interleave(heads // G, 1) for t in (case.k, case.v))
    s = torch.einsum("rhd,xhd->rhx", q.double(), k) * case.scale
    s.masked_fill_((x.cuda() >= lens.repeat_interleave(rows)[:, None])[:, None], float("-inf"))
    w = torch.softmax(s, -1)
    host = lambda t: t.cpu().numpy()
    count = host(lens.repeat_interleave(rows))
    o = {"out": host(torch.einsum("rhx,xhd->rhd", w, v)), "lse": host(torch.logsumexp(s, -1)), "count": count,
         "smax": host(torch.einsum("rhd,xhd->rhx", q.double().abs(), k.abs()).amax(-1) * case.scale),
         "mag": host(torch.einsum("rhx,xhd->rhd", w, v.abs())) + 2.0 ** -23 * count[:, None, None] * host(v.abs().max())}
    tol, lse_tol = attention_bounds(o, dim, BF16)  # (with what small weights in half floats may add, as in PackedAttentionCase)
    assert (np.abs(host(got.out.double()) - o["out"]) <= tol).all()
    assert (np.abs(host(got.lse.double()) - o["lse"]) <= lse_tol).all()


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


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 3, 20])
@pytest.mark.parametrize("base,first,later", [(25, 8.0, 16.0), (26, 8.0, 16.0), (27, 16.0, 32.0), (28, 32.0, 64.0)])
def test_huge_scores_that_rise(sv, dim, rows, base, first, later):
    """Scores (in powers of two) of 2^base + first in a history's first half, and + later in its second: there a float is a multiple
    of 4 to 32, and so are a reference and what scores may pass it by.  All of them are exact, so the weights are known."""
    n, heads, G, keys = 24, 32, 8, 1536
    case = PackedAttentionCase([keys], rows, heads, G, dim, 16)
    k = np.zeros((keys, G, dim))
    k[..., 0], k[..., 1] = 4096.0, 6144.0  # (the second of a group fixes its scale: 1024, and 1)
    k[:keys // 2, :, 16], k[keys // 2:, :, 16], k[..., 17] = 2.0, 4.0, 6.0
    x = np.arange(keys)
    slot = case.table[0][x // 16].astype(np.int64) * 16 + x % 16
    parts = list(packed.unblock(case.blocks, 16, dim))
    codes, scales, value = packed.quantize(k)
    assert np.array_equal(value, k)
    for i, new in ((0, codes), (1, scales)):
        parts[i][0].reshape(-1, G, new.shape[-1])[slot] = new
    case.blocks = packed.blocks(*parts)
    cache = case.cache(sv)
    many = sv.PackedKvCache(cache.data, cache.page_table.expand(n, -1).contiguous(), page_size=16, head_dim=dim)
    q = torch.zeros(n * rows, heads, dim, dtype=BF16, device="cuda")
    q[..., 0], q[..., 16] = 2.0 ** (base - 12), first / 2.0
    scale = np.float32(np.log(2.0))
    assert np.float32(scale * np.float32(1.4426950408889634)) == 1.0
    got = sv.paged_attention(q, many, torch.full((n,), keys, device="cuda"), max_len=rows, scale=float(scale),
                             mask=torch.zeros(n, rows, rows, dtype=torch.uint8, device="cuda"))
    w = np.where(x < keys // 2, 2.0 ** (first - later), 1.0)
    v = case.v[0].numpy().reshape(-1, G, dim)[slot].repeat(heads // G, 1)
    out, mag = np.einsum("x,xhd->hd", w, v) / w.sum(), np.einsum("x,xhd->hd", w, np.abs(v)) / w.sum()
    # the sums of 1536 weights and products in fp32, two exponentials, the weights (2^-11 of themselves) and the result rounded
    tol = (2 * keys * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -11) * mag + 2.0 ** -8 * np.abs(out)
    assert (np.abs(got.out.double().cpu().numpy() - out) <= tol).all()
    lse = (2.0 ** base + later) * np.log(2.0) + np.log(w.sum())
    assert (np.abs(got.lse.double().cpu().numpy() - lse) <= 2.0 ** -22 * lse).all()


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


@pytest.mark.parametrize("rows", [[1, 2, 1], [20, 3, 7]])
def test_rows_of_no_request_are_left(sv, rows):
    case = PackedAttentionCase([40, 300, 9], rows, 4, 2, 64, 16, ragged=True)
    n = case.q.shape[0]
    want = run(sv, case)
    case.q = torch.cat([case.q, torch.full((3, 4, 64), float("nan"), dtype=BF16)])
    out = sv.AttentionOutputs(out=torch.full((n + 3, 4, 64), 5.0, dtype=BF16, device="cuda"),
                              lse=torch.full((n + 3, 4), 5.0, device="cuda"), dev_status=torch.empty(3, dtype=torch.int32, device="cuda"))
    got = case.run(sv, out=out)
    assert torch.equal(got.out[:n], want.out) and torch.equal(got.lse[:n], want.lse)
    assert (got.out[n:] == 5.0).all() and (got.lse[n:] == 5.0).all()


@pytest.mark.parametrize("rows", [1, 20])
def test_graphs_that_share_a_workspace(sv, rows):
    """Two captured calls on one workspace, replayed by turns, with an eager one between them."""
    cases = [PackedAttentionCase(lens, rows, 8, 2, 128, 16, seed=i) for i, lens in enumerate(([3000, 40], [100, 5000]))]
    want = [run(sv, c) for c in cases]
    ws = sv.attention_workspace(2, rows, cases[0].cache(sv), 8)
    calls, graphs = [], []
    for c in cases:
        d = {"q": c.q.cuda(), "cache": c.cache(sv), "lens": torch.tensor(c.lens, device="cuda"),
             "mask": None if c.mask is None else torch.from_numpy(c.mask).cuda(),
             "slots": None if c.row_slots is None else torch.from_numpy(c.row_slots).cuda(), "scale": c.scale,
             "out": sv.AttentionOutputs.allocate(2 * rows, 8, 128, 2)}
        call = lambda d=d: sv.paged_attention(d["q"], d["cache"], d["lens"], max_len=rows, row_slots=d["slots"], mask=d["mask"],
                                              scale=d["scale"], out=d["out"], ws=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        calls.append((call, d)), graphs.append(g)
    for i in (0, 1, 1, 0):
        calls[i][1]["out"].out.fill_(7.0)
        graphs[i].replay()
        assert torch.equal(calls[i][1]["out"].out, want[i].out) and torch.equal(calls[i][1]["out"].lse, want[i].lse)
        calls[1 - i][0]()
        assert torch.equal(calls[1 - i][1]["out"].out, want[1 - i].out)


def test_calls_at_once(sv):
    """On two streams, each with a workspace of its own."""
    cases = [PackedAttentionCase([9000, 40], rows, 8, 2, 128, 16, seed=rows) for rows in (1, 20)]
    want = [run(sv, c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    made = [(c.q.cuda(), c.cache(sv), torch.tensor(c.lens, device="cuda"), sv.attention_workspace(2, c.max_len, c.cache(sv), 8)) for c in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (c, s) in enumerate(zip(cases, streams)):
            q, cache, lens, ws = made[i]
            outs[i].append(sv.paged_attention(q, cache, lens, max_len=c.max_len, scale=c.scale, ws=ws, stream=s))
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        for o in got:
            assert torch.equal(o.out, w.out) and torch.equal(o.lse, w.lse)


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("page", [1, 16, 128, 200])
def test_large_offsets(sv, rows, page):
    """Pages more than 2^32 bytes into the cache give what near ones do; a commit moves entries there."""
    free, _ = torch.cuda.mem_get_info()
    if free < 16 << 30:
        pytest.skip("needs 16 GB")
    n = 260
    need = -(-n // page)
    near = torch.arange(need, dtype=torch.int32, device="cuda")[None].contiguous()
    block = sv.PackedKvCache.block_bytes(page, 64)
    step = -(-(5 << 30) // (2 * need * 16)) * 16  # bytes from one page to the next
    g = torch.Generator(device="cuda").manual_seed(page)
    data = torch.randint(0, 256, (1, 2 * need, 2, block), dtype=torch.uint8, device="cuda", generator=g)
    parts = packed.unblock(data.cpu().numpy(), page, 64)
    for a in (parts[1], parts[3]):
        a[:] = a % 16 + 96  # moderate scales
    data = torch.from_numpy(packed.blocks(*parts)).cuda()
    far_mem = torch.zeros(2 * need * step + 2 * block, dtype=torch.uint8, device="cuda")
    far_data = torch.as_strided(far_mem, (1, 2 * need, 2, block), (0, step, block, 1))
    far_data.copy_(data)
    table = near + need
    q = torch.randn(rows, 8, 64, device="cuda", generator=g).to(BF16)
    lens = torch.tensor([n - rows], device="cuda")
    got = []
    for d in (data, far_data):
        cache = sv.PackedKvCache(d, table, page_size=page, head_dim=64)
        o = sv.paged_attention(q, cache, lens, max_len=rows)
        cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
        src = torch.tensor([(2 * need - 1) * page, need * page, 2], device="cuda")
        st = sv.kv_commit(cache, cu, src, torch.tensor([3, 4, 5], device="cuda"), max_len=3)
        got.append((o, cache.data.contiguous(), st))
    (a, ca, sa), (b, cb, sb) = got
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse) and (a.dev_status == 0).all() and (b.dev_status == 0).all()
    assert torch.equal(ca, cb) and not torch.equal(ca, data.new_zeros(1).expand_as(ca)) and sa.item() == 0 and sb.item() == 0
