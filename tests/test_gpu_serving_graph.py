"""The calls of a serving step captured in one CUDA graph and replayed on new inputs: the results of direct calls, bit for
bit."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from reject_row_vocab_gb300 import _build  # noqa: E402

_build.build()
from reject_row_vocab_gb300 import specverify as sv  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
B, PAGE, G, D, V, ROOM = 6, 16, 2, 64, 5000, 20


class _Step:
    """Attention of n rows a request, the move of the accepted ones, their log probabilities, and a gradient."""

    def __init__(self, dtype, n, heads):
        self.n, dev = n, "cuda"
        g = torch.Generator(device=dev).manual_seed(n)
        new = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
        pages = B * ROOM + B
        self.k, self.v = new(2, pages, PAGE, G, D).to(dtype), new(2, pages, PAGE, G, D).to(dtype)
        self.cache = sv.PagedKvCache(self.k, self.v, torch.randperm(pages, device=dev)[:B * ROOM].view(B, ROOM).int())
        self.q, self.logits = new(B * n, heads, D).to(dtype), new(B * n, V).to(dtype)
        self.seq_lens = torch.zeros(B, dtype=torch.int64, device=dev)
        self.ids = torch.zeros(B * n, 2, dtype=torch.int32, device=dev)
        self.cu = torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device=dev)
        self.src, self.dst = (torch.zeros(2 * B, dtype=torch.int64, device=dev) for _ in range(2))
        self.g = new(B * n, 2)
        self.out = sv.AttentionOutputs.allocate(B * n, heads, D, B, dtype)
        self.lp = sv.LogprobOutputs.allocate(B * n, 2, 5)
        self.grad, self.status = torch.empty_like(self.logits), torch.empty(B, dtype=torch.int32, device=dev)
        self.aws = sv.attention_workspace(B, n, self.cache, heads)
        self.lws = sv.logprobs_workspace(B * n, V, 5)

    def inputs(self, seed):
        g = torch.Generator().manual_seed(seed)
        lens = torch.randint(0, (ROOM - 2) * PAGE - self.n, (B,), generator=g)
        at = lens[:, None] + torch.arange(2)
        table = self.cache.page_table.cpu().long()
        self.seq_lens.copy_(lens)
        self.dst.copy_(at.reshape(-1))
        self.src.copy_((table.gather(1, (at + 16) // PAGE) * PAGE + at % PAGE).reshape(-1))
        self.ids.copy_(torch.randint(0, V, self.ids.shape, generator=g))
        self.q.copy_(torch.randn(self.q.shape, generator=g))
        self.logits.copy_(3 * torch.randn(self.logits.shape, generator=g))

    def run(self):
        sv.paged_attention(self.q, self.cache, self.seq_lens, max_len=self.n, layer=1, out=self.out, ws=self.aws)
        sv.kv_commit(self.cache, self.cu, self.src, self.dst, max_len=2, dev_status=self.status)
        sv.token_logprobs(self.logits, self.ids, top_k=5, out=self.lp, ws=self.lws)
        sv.token_logprobs_backward(self.logits, self.ids, self.lp, self.g, out=self.grad)

    def results(self):
        return [t.clone() for t in (self.out.out, self.out.lse, self.out.dev_status, self.k, self.v, self.status, self.lp.logprob,
                                    self.lp.entropy, self.lp.log_z, self.lp.top_ids, self.lp.flags, self.grad)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,heads", [(1, 8), (5, 4), (7, 16)])
def test_a_captured_step_repeats_direct_calls(dtype, n, heads):
    step = _Step(dtype, n, heads)
    step.inputs(0)
    step.run()  # (what is set up once is set up before the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for seed in range(1, 5):
        step.inputs(seed)
        k, v = step.k.clone(), step.v.clone()
        step.run()
        direct = step.results()
        step.k.copy_(k)
        step.v.copy_(v)
        for t in (step.out.out, step.out.lse, step.lp.logprob, step.grad):
            t.fill_(7.0)
        graph.replay()
        for a, b in zip(direct, step.results()):
            assert torch.equal(a, b)
        assert int(step.out.dev_status.abs().sum()) == 0 and int(step.status.abs().sum()) == 0
