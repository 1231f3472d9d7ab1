"""The KV commit in the 4-bit cache, and a serving step on it: rows appended, attended to, committed, read back; in a CUDA
graph and on another stream."""
import numpy as np
import pytest
import torch

from oracle import packed, serving
from tests.packed_cases import AppendCase, check_append
from tests.serving_cases import BF16, F32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    from reject_row_vocab_gb300 import specverify
    return specverify


def commit_case(batch, rows, layers, heads, dim, page, length, in_place=False, seed=0):
    rng = np.random.default_rng(seed)
    need = -(-(length + rows + 1) // page)
    spare = -(-batch * rows // page)
    pages = batch * need + spare
    order = rng.permutation(pages)
    table = order[:batch * need].reshape(batch, need).astype(np.int32)
    stage = (order[batch * need:, None] * page + np.arange(page)).reshape(-1)[:batch * rows].reshape(batch, rows)
    cu, src, dst = [0], [], []
    for b in range(batch):
        n = int(rng.integers(0, rows + 1))
        pick = np.sort(rng.choice(rows, n, replace=False))
        for k, j in enumerate(pick):
            x = length + j
            src.append(table[b, x // page] * page + x % page if in_place else stage[b, j])
            dst.append(length + k)
        cu.append(len(src))
    data = rng.integers(0, 256, (layers, pages, heads, packed.block_bytes(page, dim)), dtype=np.uint8)
    return table, np.array(cu, np.int32), np.array(src, np.int64), np.array(dst, np.int64), data


@pytest.mark.parametrize("batch,rows,layers,heads,dim,page,length,in_place", [
    (1, 5, 4, 8, 128, 16, 30, False), (9, 16, 3, 2, 64, 16, 100, True), (3, 7, 2, 1, 256, 1, 5, True), (4, 60, 2, 4, 96, 5, 11, True),
    (2, 33, 5, 3, 32, 8, 0, False), (5, 4, 40, 2, 160, 64, 63, True), (1, 600, 1, 2, 64, 16, 3, True), (2, 9, 2, 2, 224, 3, 4, True)])
def test_commit(sv, batch, rows, layers, heads, dim, page, length, in_place):
    table, cu, src, dst, data = commit_case(batch, rows, layers, heads, dim, page, length, in_place)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    cache = sv.PackedKvCache(dev(data), dev(table), page_size=page, head_dim=dim)
    status = sv.kv_commit(cache, dev(cu), dev(src), dev(dst), max_len=rows)
    parts = packed.unblock(data, page, dim)
    moved = [serving.kv_commit(p, table, cu, src, dst, rows) for p in parts]
    got = packed.unblock(cache.data.cpu().numpy(), page, dim)
    for g, (want, st) in zip(got, moved):
        assert np.array_equal(g, want) and np.array_equal(status.cpu().numpy().view(np.uint32), st)


def test_commit_reports_bad_entries(sv):
    table, cu, src, dst, data = commit_case(4, 6, 2, 2, 64, 4, 9, seed=3)
    cu = np.array([0, 2, 4, 3, 5], np.int32)
    src, dst = src[:5].copy(), np.array([9, 10, 9, 10 ** 9, 9])
    src[0] = -1
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    cache = sv.PackedKvCache(dev(data), dev(table), page_size=4, head_dim=64)
    status = sv.kv_commit(cache, dev(cu), dev(src), dev(dst), max_len=6)
    parts = packed.unblock(data, 4, 64)
    moved = [serving.kv_commit(p, table, cu, src, dst, 6) for p in parts]
    for g, (want, st) in zip(packed.unblock(cache.data.cpu().numpy(), 4, 64), moved):
        assert np.array_equal(g, want) and np.array_equal(status.cpu().numpy().view(np.uint32), st)


class Step:
    """A layer's step of a draft tree: append, attention, commit of an accepted path, and reading the history back."""

    def __init__(self, sv, is_packed, seed=0):
        self.case = AppendCase([30, 0, 200], 6, 8, 2, 64, 16, BF16, is_packed=is_packed, staged=True, seed=seed)
        c = self.case
        c.table = np.concatenate([c.table, np.arange(3)[:, None].astype(np.int32) + c.pages], 1)  # room for committed rows
        if is_packed:
            c.before = np.concatenate([c.before, c.before[:, :3]], 1)
        else:
            c.before = [torch.cat([t, t[:, :3]], 1) for t in c.before]
        c.pages += 3
        rng = np.random.default_rng(seed)
        used = [-(-n // 16) for n in c.lens]
        for b in range(3):  # the page behind the history
            c.table[b, used[b]] = c.pages - 3 + b
        if is_packed:  # bytes that stand for moderate numbers
            parts = packed.unblock(c.before, 16, 64)
            for a in (parts[1], parts[3]):
                a[:] = rng.integers(96, 112, a.shape)
            c.before = packed.blocks(*parts)
        c.positions = np.array([n + d for n in c.lens for d in (0, 1, 1, 2, 2, 3)])
        par = [-1, 0, 0, 1, 2, 3]
        mask = np.zeros((6, 6), np.uint8)
        for i in range(6):
            j = i
            while j >= 0:
                mask[i, j] = 1
                j = par[j]
        self.mask = torch.from_numpy(np.repeat(mask[None], 3, 0)).cuda()
        self.d = c.make(sv)
        dev = dict(device="cuda")
        path = [0, 1, 3, 5]
        self.cu = torch.tensor([0, 4, 8, 12], dtype=torch.int32, **dev)
        self.src = torch.tensor([int(c.row_slots[b * 6 + j]) for b in range(3) for j in path], **dev)
        self.dst = torch.tensor([c.lens[b] + k for b in range(3) for k in range(4)], **dev)
        self.out = sv.KvAppendOutputs.allocate(18, 8, 64, 3)
        self.attn = sv.AttentionOutputs.allocate(18, 8, 64, 3)
        self.ws = sv.attention_workspace(3, 6, self.d["cache"], 8)
        self.status = torch.zeros(3, dtype=torch.int32, **dev)
        self.back = sv.KvReadOutputs.allocate(12, 2, 64, 3)

    def run(self, sv, stream=None):
        d = self.d
        self.case.append(sv, d, out=self.out, stream=stream)
        sv.paged_attention(self.out.q, d["cache"], d["seq_lens"], max_len=6, row_slots=d["slots"], mask=self.mask, out=self.attn,
                           ws=self.ws, stream=stream)
        sv.kv_commit(d["cache"], self.cu, self.src, self.dst, max_len=6, dev_status=self.status, stream=stream)
        sv.kv_read(d["cache"], layer=0, seq_lens=d["seq_lens"], cu_seqlens=self.cu, max_len=6, out=self.back, stream=stream)
        return [t.clone() for t in (self.out.q, self.attn.out, self.attn.lse, self.back.k, self.back.v)]

    def check(self, results):
        """Against the oracle on what the cache holds."""
        c, d = self.case, self.d
        q, out, lse, k, v = results
        if c.is_packed:
            parts = packed.unblock(d["data"].cpu().numpy(), 16, 64)
            held = [packed.values(parts[i], parts[i + 1])[0] for i in (0, 2)]
        else:
            held = [d[n][0].double().cpu().numpy() for n in ("k", "v")]
        o = serving.attention(q.double().cpu().numpy(), *held, c.table, c.lens, [0, 6, 12], [6] * 3, 64 ** -0.5, c.row_slots,
                              self.mask.cpu().numpy())
        # weights and outputs rounded to bf16, as the attention tests derive it; fp32 sums of 230 keys are far below that
        tol = 2.0 ** -8 * (o["mag"] + np.abs(o["out"])) + 2.0 ** -12 * o["mag"]
        assert (np.abs(out.double().cpu().numpy() - o["out"]) <= tol).all()
        slot = [int(c.table[b][x // 16]) * 16 + x % 16 for b in range(3) for x in range(c.lens[b], c.lens[b] + 4)]
        staged = self.src.cpu().numpy()
        for have, h in zip((k, v), held):
            flat = h.reshape(-1, 2, 64)
            assert np.array_equal(have.double().cpu().numpy(), flat[slot]) and np.array_equal(flat[slot], flat[staged])
        assert (self.out.dev_status == 0).all() and (self.attn.dev_status == 0).all() and (self.status == 0).all()


@pytest.mark.parametrize("is_packed", [False, True])
def test_a_serving_step(sv, is_packed):
    s = Step(sv, is_packed)
    s.check(s.run(sv))
    o = s.case.oracle()
    assert (o["slot"] >= 0).all()


@pytest.mark.parametrize("is_packed", [False, True])
def test_a_step_in_a_graph_and_on_another_stream(sv, is_packed):
    s = Step(sv, is_packed)
    want = s.run(sv)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = s.run(sv, stream=stream)
    stream.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = s.run(sv)
    for seed in (1, 2):
        fresh = Step(sv, is_packed, seed)
        s.d["qkv"].copy_(fresh.d["qkv"])
        g.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in kept]
        for a, b in zip(replayed, s.run(sv)):
            assert torch.equal(a, b)
        s.check(replayed)
