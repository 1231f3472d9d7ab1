"""Token log probabilities, entropy, top alternatives and their gradient against the fp64 oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from oracle import serving  # noqa: E402
from reject_row_vocab_gb300 import _build  # noqa: E402

_build.build()
from reject_row_vocab_gb300 import device_workload as dw  # noqa: E402
from reject_row_vocab_gb300 import specverify as sv  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def _logits(rows, V, dtype, seed, sigma=3.0):
    g = torch.Generator().manual_seed(seed)
    return (sigma * torch.randn(rows, V, generator=g)).to(dtype)


def _tolerances(o, V, T):
    """A term of Z costs its exponential (2^-21) and its exponent's rounding; a thread sums V / 256 terms and the block
    a few more, each 2^-24; a difference over T rounds twice."""
    sums = (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -20
    lz = sums * (1 + o["spread"]) + 2.0 ** -23 * np.where(np.isfinite(o["log_z"]), np.abs(o["log_z"]), 0)
    ent = lz + sums * (1 + o["spread"]) ** 2
    return lz, ent


def _check(logits, ids, temp=None, top_k=0, row_index=None, **kw):
    up = lambda a, t: None if a is None else torch.tensor(np.asarray(a), dtype=t).cuda()
    d = dw.padded_rows(logits, "cuda")
    got = sv.token_logprobs(d, up(ids, torch.int32), top_k=top_k, row_index=up(row_index, torch.int32),
                            row_temp=up(temp, F32), **kw)
    o = serving.logprobs(logits.double().numpy(), np.asarray(ids), None if temp is None else np.float32(temp), top_k,
                         row_index)
    lz, ent = _tolerances(o, logits.shape[1], temp)
    num = lambda t: t.double().cpu().numpy()
    assert np.array_equal(num(got.row_max), o["row_max"])
    assert np.array_equal(got.flags.cpu().numpy().view(np.uint32), o["flags"])
    for name, tol in (("log_z", lz), ("entropy", ent)):
        x, fine = num(getattr(got, name)), np.isfinite(o[name])
        assert np.array_equal(x[~fine], o[name][~fine])
        assert (np.abs(x[fine] - o[name][fine]) <= tol[fine]).all(), (name, (np.abs(x[fine] - o[name][fine]) / tol[fine]).max())
    names = ["logprob"] + (["top_logprob"] if top_k else [])
    for name in names:
        with np.errstate(over="ignore"):  # a log probability beyond fp32's range is -inf in fp32
            o[name] = np.where(np.isneginf(o[name].astype(np.float32)), -np.inf, o[name])
        x, fine = num(getattr(got, name)), np.isfinite(o[name])
        tol = lz[:, None] + 2.0 ** -22 * np.abs(np.where(fine, o[name], 0))
        assert np.array_equal(x[~fine], o[name][~fine]), name
        assert (np.abs(x[fine] - o[name][fine]) <= tol[fine]).all(), name
    if top_k:
        assert np.array_equal(got.top_ids.cpu().numpy(), o["top_ids"])
    return got, o


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,V", [(1, 1), (2, 3), (3, 7), (2, 8), (5, 9), (4, 255), (3, 1000), (2, 8191), (3, 32003),
                                    (1, 151936), (700, 257)])
@pytest.mark.parametrize("top_k", [0, 1, 20, 64])
def test_sizes(dtype, rows, V, top_k):
    rng = np.random.default_rng(V)
    _check(_logits(rows, V, dtype, V), rng.integers(0, V, (rows, 2)), top_k=top_k)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("temp", [0.0, 1e-31, 1e-6, 0.3, 1.0, 7.5, 1e6, INF, -1.0, float("nan")])
def test_temperatures(dtype, temp):
    rng = np.random.default_rng(2)
    _check(_logits(6, 5003, dtype, 8), rng.integers(0, 5003, (6, 3)), temp=[temp] * 6, top_k=5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [50, 5000, 70001])
def test_equal_logits_resolve_to_the_lowest_ids(dtype, V):
    rng = np.random.default_rng(V)
    x = torch.zeros(4, V)
    x[1] = 2.5
    x[2] = torch.from_numpy(rng.integers(-2, 3, V).astype(np.float32))
    x[3] = torch.from_numpy(np.where(rng.integers(0, 2, V) == 1, 0.0, -0.0).astype(np.float32))
    _check(x.to(dtype), rng.integers(0, V, (4, 1)), top_k=20)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [40, 4096, 40009])
def test_masked_and_unusable_logits(dtype, V):
    x = _logits(8, V, dtype, V)
    low = torch.finfo(dtype).min
    x[0] = -INF                      # nothing left
    x[1, 1:] = -INF                  # one token left
    x[2, ::2] = -INF
    x[3, 5:] = low                   # masked with the type's lowest value
    x[4, 3], x[4, V - 1], x[4, 20] = float("nan"), INF, -INF
    x[5] = INF                       # nothing usable
    x[6] = low                       # every token at the lowest value: uniform
    x[7, : V // 2] = -INF
    ids = np.stack([np.zeros(8, int), np.full(8, 3), np.full(8, V - 1), np.full(8, -1), np.full(8, V), np.full(8, -2)], 1)
    _check(x, ids, top_k=6)
    _check(x, ids, top_k=6, temp=[0.5] * 8)
    _check(x, ids, top_k=0, temp=[1e30] * 8)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sorted_rows(dtype):
    # rising and falling rows, and the largest values packed into one thread's columns
    V = 60000
    x = torch.linspace(-20, 20, V).repeat(4, 1)
    x[1] = x[1].flip(0)
    x[2] = -10.0
    x[2, 8 * 256 * torch.arange(28)] = torch.arange(28).float()
    x[3] = -10.0
    x[3, 100:170] = torch.arange(70).float()
    _check(x.to(dtype), np.full((4, 1), 3), top_k=64)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_row_index(dtype):
    x = _logits(9, 3001, dtype, 4)
    idx = [3, -1, 3, 8, 0, 9, -2, 7]
    rng = np.random.default_rng(5)
    _check(x, rng.integers(0, 3001, (8, 2)), row_index=idx, top_k=4, temp=rng.uniform(0.5, 1.5, 8))


def test_no_ids_and_strided_ids():
    x = _logits(4, 1000, F32, 6)
    _check(x, np.zeros((4, 0), int), top_k=3)
    d = dw.padded_rows(x, "cuda")
    wide = torch.randint(0, 1000, (4, 6), dtype=torch.int32, device="cuda")
    a = sv.token_logprobs(d, wide[:, :2])
    b = sv.token_logprobs(d, wide[:, :2].contiguous())
    assert torch.equal(a.logprob, b.logprob)
    assert torch.equal(sv.token_logprobs(d, wide[:, 0].contiguous()).logprob, a.logprob[:, :1])


def test_repeats_are_bit_equal_and_one_workspace_serves_all_sizes():
    ws = sv.logprobs_workspace(1, 8, 64)
    first = {}
    for rep in range(2):
        for rows, V, k in ((3, 151936, 64), (300, 40000, 5), (1, 20000, 0), (64, 151936, 20)):
            x = dw.padded_rows(_logits(rows, V, BF16, rows), "cuda")
            ids = torch.zeros(rows, 1, dtype=torch.int32, device="cuda")
            o = sv.token_logprobs(x, ids, top_k=k, ws=ws)
            key = (rows, V, k)
            if rep:
                for a, b in zip(first[key], (o.logprob, o.entropy, o.log_z, o.top_ids)):
                    assert a is b is None or torch.equal(a, b)
            first[key] = (o.logprob, o.entropy, o.log_z, o.top_ids)


def test_committed_tokens_of_a_verification():
    # accept_rows and out_tokens of a verify call, as they come
    from reject_row_vocab_gb300 import workload as wl
    w = wl.rejection_chain(batch=6, m=4, vocab=2048, dtype="bf16", seed=3, name="logprobs_of_commits")
    d = dw.DeviceInputs.from_workload(w)
    o = dw.run(w, d)
    lp = sv.token_logprobs(d["logits"], o.out_tokens.view(-1), row_index=o.accept_rows.view(-1))
    full = torch.log_softmax(d["logits"].float(), 1)
    rows, toks = o.accept_rows.view(-1).long(), o.out_tokens.view(-1).long()
    live = rows >= 0
    want = torch.where(live, full[rows.clamp(min=0), toks.clamp(min=0)], torch.zeros((), device="cuda"))
    assert (lp.logprob[:, 0] - want).abs().max() < 1e-4
    assert (lp.logprob[~live] == 0).all() and (lp.flags == 0).all()


# ---- gradient


def _grad(logits, ids, g, temp=None, g_ent=None, top_k=0, g_top=None):
    up = lambda a, t: None if a is None else torch.tensor(np.asarray(a), dtype=t).cuda()
    d = dw.padded_rows(logits, "cuda")
    kept = sv.token_logprobs(d, up(ids, torch.int32), top_k=top_k, row_temp=up(temp, F32))
    out = sv.token_logprobs_backward(d, up(ids, torch.int32), kept, up(g, F32), g_entropy=up(g_ent, F32),
                                     g_top=up(g_top, F32), row_temp=up(temp, F32))
    top = kept.top_ids.cpu().numpy() if top_k else None
    want, mag = serving.logprobs_grad(logits.double().numpy(), np.asarray(ids), np.float32(g),
                                      None if temp is None else np.float32(temp),
                                      None if g_ent is None else np.float32(g_ent), top,
                                      None if g_top is None else np.float32(g_top))
    got = out.double().cpu().numpy()
    # each term carries its probability's error (its exponent's rounding, the log sum's, an exponential), then one rounding
    V = logits.shape[1]
    tol = mag * ((V / 256 + 64) * 2.0 ** -24 + 2.0 ** -18) + 1e-37
    if logits.dtype == BF16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,V", [(1, 1), (2, 3), (3, 9), (5, 1000), (2, 32003), (400, 513), (1, 151936)])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient_sizes(dtype, rows, V, entropy):
    rng = np.random.default_rng(V)
    _grad(_logits(rows, V, dtype, V), rng.integers(0, V, (rows, 3)), rng.normal(size=(rows, 3)),
          temp=rng.uniform(0.4, 2.0, rows), g_ent=rng.normal(size=rows) if entropy else None, top_k=4,
          g_top=rng.normal(size=(rows, 4)))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradient_of_masked_padded_and_repeated_tokens(dtype):
    V = 3001
    x = _logits(6, V, dtype, 3)
    x[0] = -INF
    x[1, 2:] = -INF
    x[2, 4], x[2, 7] = float("nan"), INF
    x[3, 10:] = torch.finfo(dtype).min
    rng = np.random.default_rng(3)
    ids = rng.integers(0, V, (6, 5))
    ids[:, 1] = ids[:, 0]
    ids[:, 2] = [-1, 0, 4, 3, V, -9]
    ids[2, 3] = 7
    _grad(x, ids, rng.normal(size=(6, 5)), g_ent=rng.normal(size=6))
    _grad(x, ids, rng.normal(size=(6, 5)), temp=[0.0, 0.5, 1e-31, 2.0, 1.0, 0.7])


def test_gradient_against_differences():
    # central differences of the definition in 64 bits
    rng = np.random.default_rng(7)
    V = 37
    x = _logits(3, V, F32, 5)
    ids, g, ge, T = rng.integers(0, V, (3, 2)), np.float32(rng.normal(size=(3, 2))), np.float32(rng.normal(size=3)), [0.7, 1.3, 1.0]
    got = _grad(x, ids, g, temp=T, g_ent=ge)
    base = x.double().numpy()
    h = 1e-5

    def loss(l):
        o = serving.logprobs(l, ids, np.float32(T))
        return (o["logprob"] * g).sum() + (o["entropy"] * ge).sum()
    for i in range(3):
        for v in range(V):
            a, b = base.copy(), base.copy()
            a[i, v] += h
            b[i, v] -= h
            # truncation h^2, cancellation 1e-15 / h, and fp32 results
            assert abs((loss(a) - loss(b)) / (2 * h) - got[i, v]) < 2e-5


def test_gradient_in_a_strided_output_leaves_its_padding():
    x = dw.padded_rows(_logits(3, 1001, BF16, 9), "cuda")
    ids = torch.tensor([[5], [1000], [7]], dtype=torch.int32, device="cuda")
    kept = sv.token_logprobs(x, ids)
    buf = torch.full((3, 1024), 9.0, dtype=BF16, device="cuda")
    g = torch.ones(3, 1, device="cuda")
    sv.token_logprobs_backward(x, ids, kept, g, out=buf[:, :1001])
    assert (buf[:, 1001:] == 9.0).all()
    assert torch.equal(buf[:, :1001], sv.token_logprobs_backward(x, ids, kept, g))


def test_gradient_refuses_to_overwrite_the_logits():
    x = dw.padded_rows(_logits(3, 1000, BF16, 9), "cuda")
    ids = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    kept = sv.token_logprobs(x, ids)
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.token_logprobs_backward(x, ids, kept, torch.ones(3, 1, device="cuda"), out=x)
    assert e.value.code == 5
