"""Rounds of tree speculative decoding with a toy model of one attention layer, all on the library's calls.

Each round: a draft head proposes a tree a request; `kv_append` puts the rows' keys and values into staged slots of the paged
cache; `paged_attention` gives the verify rows' attention under the tree's mask; `greedy_tree` accepts a path; `kv_commit`
moves the accepted rows' keys and values into place; `token_logprobs` gives the committed tokens' log probabilities with the
most likely alternatives; and the draft head takes a step on the committed tokens, its gradient from `token_logprobs_backward`.

    python examples/tree_round.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from reject_row_vocab_gb300 import specverify as sv  # noqa: E402

PARENTS = [-1, 0, 0, 1, 1, 2, 3]  # anchor, two guesses, two behind the first, one behind the second, one more step


class ToyModel:
    """x = token + position embedding, one layer of grouped-query attention, logits = (x + attention) @ head."""

    def __init__(self, vocab=1000, width=128, heads=8, kv_heads=2, dim=64, positions=256, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        mat = lambda *s: (torch.randn(*s, generator=g) / s[0] ** 0.5).to(device)  # noqa: E731
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.embed, self.place = mat(vocab, width) * 30, mat(positions, width) * 8
        self.q, self.k, self.v = mat(width, heads * dim), mat(width, kv_heads * dim), mat(width, kv_heads * dim)
        self.o, self.head = mat(heads * dim, width), mat(width, vocab)

    def hidden(self, tokens, positions):
        return self.embed[tokens] + self.place[positions]

    def qkv(self, x):
        n = x.shape[0]
        return ((x @ self.q).view(n, self.heads, self.dim), (x @ self.k).view(n, self.kv_heads, self.dim),
                (x @ self.v).view(n, self.kv_heads, self.dim))


def run(prompts, rounds=8, vocab=1000, page=16, top_k=3, lr=0.5, seed=0, device="cuda"):
    """prompts: a list of token lists.  Returns each request's generated tokens, their log probabilities, the mean accepted
    drafts of each round, and the draft head's losses."""
    m = ToyModel(vocab=vocab, seed=seed, device=device)
    B, N = len(prompts), len(PARENTS)
    room = -(-(max(map(len, prompts)) + rounds * N) // page)  # pages a request can need
    pages = B * room + -(-B * N // page)                      # and the staged rows' pages behind them
    k = torch.zeros(1, pages, page, m.kv_heads, m.dim, device=device)
    v = torch.zeros_like(k)
    order = torch.randperm(B * room, generator=torch.Generator().manual_seed(seed))
    cache = sv.PagedKvCache(k, v, order.to(torch.int32).view(B, room).to(device))
    row_slots = torch.arange(B * N, device=device) + B * room * page

    # the prompts' keys and values, all but the last token, which is the first anchor
    lens = [len(p) - 1 for p in prompts]
    ids = torch.tensor([t for p in prompts for t in p[:-1]], device=device, dtype=torch.long)
    at = torch.tensor([i for n in lens for i in range(n)], device=device, dtype=torch.long)
    cu = torch.tensor([sum(lens[:b]) for b in range(B + 1)], dtype=torch.int32, device=device)
    _, kk, vv = m.qkv(m.hidden(ids, at))
    filled = sv.kv_append(cache, kk, vv, seq_lens=torch.zeros(B, dtype=torch.int64, device=device), cu_seqlens=cu,
                          max_len=max(lens + [1]))
    seq_lens = torch.tensor(lens, dtype=torch.int64, device=device)
    anchor = torch.tensor([p[-1] for p in prompts], device=device)

    parents = torch.tensor([PARENTS] * B, dtype=torch.int32, device=device)
    draft_head = m.head.clone()
    attn_out = sv.AttentionOutputs.allocate(B * N, m.heads, m.dim, B, torch.float32, device)
    attn_ws = sv.attention_workspace(B, N, cache, m.heads)
    verify_ws = sv.workspace(B * N, B, vocab, N, device)
    logp_ws = sv.logprobs_workspace(B * N, vocab, top_k, device)
    tokens_of, logprobs_of, accepted, losses = [[] for _ in range(B)], [[] for _ in range(B)], [], []
    for _ in range(rounds):
        tree = sv.build_tree(parents, seq_lens)
        # the draft: each node's guesses are the likeliest tokens behind its own, without attention
        tokens = torch.empty(B, N, dtype=torch.int32, device=device)
        tokens[:, 0] = anchor
        for node in range(1, N):
            up = PARENTS[node]
            guess = (m.hidden(tokens[:, up].long(), tree["positions"][:, up]) @ draft_head).topk(2).indices
            tokens[:, node] = guess[:, PARENTS[:node].count(up)]
        x = m.hidden(tokens.view(-1).long(), tree["positions"].view(-1))
        q, kk, vv = m.qkv(x)
        sv.kv_append(cache, kk, vv, seq_lens=seq_lens, max_len=N, row_slots=row_slots, out=filled)

        sv.paged_attention(q, cache, seq_lens, max_len=N, row_slots=row_slots, mask=tree["mask"], out=attn_out, ws=attn_ws)
        logits = (x + attn_out.out.view(B * N, -1) @ m.o) @ m.head
        done = sv.greedy_tree(logits, tokens, parents, first_child=tree["first_child"], next_sibling=tree["next_sibling"],
                              row_slots=row_slots, seq_lens=seq_lens, ws=verify_ws)
        status = sv.kv_commit(cache, done.commit_cu, done.commit_src_slot, done.commit_dst_pos, max_len=N)
        new = done.out_tokens.view(-1)
        rows = done.accept_rows.view(-1)
        lp = sv.token_logprobs(logits, new, top_k=top_k, row_index=rows, ws=logp_ws)

        # a step of the draft head on the committed tokens (rows that are padding have token -1, and no part)
        xd = x[rows.clamp(min=0).long()]
        draft = xd @ draft_head
        kept = sv.token_logprobs(draft, new)
        count = done.num_out.sum()
        grad = sv.token_logprobs_backward(draft, new, kept, -torch.ones(B * N, 1, device=device) / count)
        draft_head -= lr * xd.t() @ grad / xd.square().sum(1).mean()
        losses.append(float(-kept.logprob.sum() / count))

        bits = torch.cat([filled.dev_status, status, attn_out.dev_status, done.dev_status, lp.flags])
        assert int(bits.abs().sum()) == 0, "data errors"
        for b, n in enumerate(done.num_out.tolist()):
            tokens_of[b] += done.out_tokens[b, :n].tolist()
            logprobs_of[b] += lp.logprob.view(B, N)[b, :n].tolist()
        accepted.append(float(done.accept_len.float().mean()))
        seq_lens = seq_lens + done.num_out
        anchor = done.bonus.long()
    return tokens_of, logprobs_of, accepted, losses


if __name__ == "__main__":
    gen = torch.Generator().manual_seed(1)
    got = run([torch.randint(1000, (n,), generator=gen).tolist() for n in (5, 40, 17, 1)])
    print("accepted drafts a round:", ["%.2f" % a for a in got[2]])
    print("draft loss a round:     ", ["%.3f" % x for x in got[3]])
    for toks, lps in zip(got[0], got[1]):
        print(len(toks), "tokens, mean log probability %.3f:" % (sum(lps) / len(lps)), toks[:12], "...")
