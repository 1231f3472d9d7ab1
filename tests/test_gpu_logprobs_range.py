"""Token log probabilities over the whole range of logits and temperatures: masks of any finite value, the smallest
temperatures that are sampled, the largest logits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from test_gpu_logprobs import BF16, F32, _check, _grad, _logits, dw, sv  # noqa: E402

MASKS = [-1e4, -65504.0, -1e8, -1e9, -1e10, -1e12, -1e20, -1e30, -3e38]


def _masked(V, low, dtype):
    """Rows masked with `low`: wholly, but for one token, in their first and second half, every other token, at random, and
    by adding it."""
    x = _logits(8, V, F32, V)
    keep = torch.zeros(8, V, dtype=torch.bool)
    keep[1, V - 2] = True
    keep[2, V // 2:] = True
    keep[3, : V // 2] = True
    keep[4, ::2] = True
    keep[5] = torch.rand(V, generator=torch.Generator().manual_seed(1)) < 0.01
    keep[6, 3] = True
    added = x[7] + low
    x = torch.where(keep, x, torch.tensor(low))
    x[7] = added
    x[7, V // 3] = 1.5
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("low", MASKS)
@pytest.mark.parametrize("temp", [1.0, 0.3, 0.1])
def test_finite_masks(dtype, low, temp):
    for V in (700, 20011):
        ids = np.stack([np.full(8, 3), np.full(8, V - 2), np.full(8, V // 3)], 1)
        _check(_masked(V, low, dtype), ids, temp=[temp] * 8, top_k=5)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_finite_masks_of_rows_that_several_blocks_share(dtype):
    V = 151936
    for low in (-1e10, -1e30):
        _check(_masked(V, low, dtype), np.full((8, 1), V // 3), top_k=20)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("temp", [1e-7, 1e-8, 1e-9, 1e-10, 1e-12, 1e-20, 2e-30])
@pytest.mark.parametrize("sigma", [0.01, 3.0, 1e4])
def test_smallest_temperatures(dtype, temp, sigma):
    rng = np.random.default_rng(2)
    x = _logits(5, 20011, dtype, 8, sigma)
    x[1] = x[1, 0]                          # all equal
    x[2, 7] = x[2, 19000] = x[2].max() * 2  # two tokens share the first place
    _check(x, rng.integers(0, 20011, (5, 3)), temp=[temp] * 5, top_k=5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("temp", [2e-30, 1e-12, 1.0, 1e6])
def test_largest_logits(dtype, temp):
    x = _logits(4, 5003, F32, 3).clamp(-8, 8) * 2e37
    x[1] = x[1].abs()
    x[2] = -x[2].abs()
    x[3, ::3] = 0.0
    _check(x.to(dtype), np.full((4, 2), 3), temp=[temp] * 4, top_k=5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("low", [-1e9, -1e10, -1e30])
@pytest.mark.parametrize("temp", [1.0, 0.1])
def test_gradient_of_masked_rows(dtype, low, temp):
    V = 3001
    rng = np.random.default_rng(4)
    _grad(_masked(V, low, dtype), rng.integers(0, V, (8, 2)), rng.normal(size=(8, 2)), temp=[temp] * 8,
          g_ent=rng.normal(size=8))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("temp", [1e-8, 1e-12, 1e-20])
def test_gradient_at_the_smallest_temperatures(dtype, temp):
    rng = np.random.default_rng(5)
    x = _logits(4, 3001, dtype, 6)
    _grad(x, rng.integers(0, 3001, (4, 2)), rng.normal(size=(4, 2)), temp=[temp] * 4)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("temp", [0.3, 0.1, 0.05])
def test_gradient_of_probabilities_at_the_end_of_fp32(dtype, temp):
    rng = np.random.default_rng(6)
    _grad(_logits(8, 20011, dtype, 9), rng.integers(0, 20011, (8, 2)), rng.normal(size=(8, 2)), temp=[temp] * 8,
          g_ent=rng.normal(size=8))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_small_weights_beside_large_ones(dtype):
    # 256 tokens of weight 1, one early in each of the sums that 128 threads hold, and 151680 of 2^-24.9, each below the last
    # place of a sum that has one of the others; every row in one block
    V, n = 151936, 1024
    x = torch.full((1, V), -17.25)
    per = 8 if dtype == BF16 else 4
    x[0, (per * torch.arange(128)[:, None] + torch.arange(2)).ravel()] = 0.0
    d = dw.padded_rows(x.to(dtype), "cuda")
    got = sv.token_logprobs(d, torch.zeros(n, 1, dtype=torch.int32, device="cuda"),
                            row_index=torch.zeros(n, dtype=torch.int32, device="cuda"))
    rest = 151680 * np.exp(-17.25)
    want = np.log(256 + rest)
    # a sum's 64 elements, the ten such sums of a row, and the join of 128 threads, each 2^-24; an exponential 2^-21
    tol = (64 + 10 + 64) * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -23 * want
    assert (got.log_z.double().cpu() - want).abs().max() <= tol
    entropy = want + 17.25 * rest / (256 + rest)
    assert (got.entropy.double().cpu() - entropy).abs().max() <= tol * (1 + 17.25)
