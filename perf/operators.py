"""What the serving-side operators are measured on: paged attention of the verify rows, the KV commit, and the log
probabilities of given tokens with their gradient.

`run` computes each operator in its plain form (elementary torch operations in 32 bits), or, where `own` is true,
through the library's public entry points.  Lengths, trees and accepted counts are functions of the case alone, so that
`work` can count them; values come from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GOLDEN = 0.6180339887498949


# ----------------------------------------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------------------------------------


def _attn(name, batch, rows, lo, hi, heads, kv_heads, head_dim, page, dtype="bf16", ragged=False, tree=False,
          staged=False):
    c = {"op": "attn", "batch": batch, "rows": rows, "lo": lo, "hi": hi, "heads": heads, "kv_heads": kv_heads,
         "head_dim": head_dim, "page": page, "dtype": dtype, "ragged": ragged, "tree": tree, "staged": staged}
    return dict(c, name=name) if name else c


def _logp(name, rows, vocab, dtype, ids, top, temp, live, masked):
    c = {"op": "logp", "rows": rows, "vocab": vocab, "dtype": dtype, "ids": ids, "top": top, "temp": temp,
         "live": live, "masked": masked}
    return dict(c, name=name) if name else c


def _grad(name, rows, vocab, dtype, ids, top, temp, entropy):
    c = {"op": "grad", "rows": rows, "vocab": vocab, "dtype": dtype, "ids": ids, "top": top, "temp": temp,
         "entropy": entropy}
    return dict(c, name=name) if name else c


def _commit(name, batch, rows, layers, kv_heads, head_dim, page, length, dtype="bf16"):
    c = {"op": "commit", "batch": batch, "rows": rows, "layers": layers, "kv_heads": kv_heads, "head_dim": head_dim,
         "page": page, "length": length, "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request decoding one token a step over a short history: a chat's first answer, where latency counts
        _attn("attn_decode_small", 1, 1, 500, 500, 32, 8, 128, 16),
        # a full decoding batch with histories of very different lengths, one token each
        _attn("attn_decode_batch", 128, 1, 64, 8192, 32, 8, 128, 16),
        # a 64-request block of 16 rows (anchor and 15 drafts) a request, drafts in place behind the history
        _attn("attn_verify_block", 64, 16, 100, 4000, 32, 8, 128, 64),
        # 16 requests' draft trees of 17 nodes, a pool of single slots, the drafts' K/V staged elsewhere in the pool
        _attn("attn_verify_tree", 16, 17, 37, 2100, 16, 2, 128, 1, tree=True, staged=True),
        # two requests of a long document, 5 rows each: few rows, so the length is split over the whole GPU
        _attn("attn_long_chain", 2, 5, 60000, 100000, 32, 4, 128, 32),
        # a small model kept in fp32, ragged verify lengths of 1..8
        _attn("attn_ragged_f32", 24, 8, 1, 900, 8, 4, 64, 16, dtype="f32", ragged=True),
        # one request's 5 rows over a 32000-token vocabulary in fp32, the chosen token and 5 alternatives a row
        _logp("logp_chain", 5, 32000, "f32", 1, 5, False, 1.0, 0),
        # a full block's rows, bf16, a temperature each, the chosen token and 20 alternatives
        _logp("logp_block", 1024, 151936, "bf16", 1, 20, True, 1.0, 0),
        # draft training on a block's rows: the gradient of the tokens' log probabilities and of an entropy term
        _grad("grad_block", 1024, 151936, "bf16", 1, 0, False, True),
        # a small fp32 head, odd vocabulary: gradient of 4 given tokens and 5 alternatives a row, as a distillation loss
        _grad("grad_distill", 80, 32003, "f32", 4, 5, True, False),
        # one request's accepted chain moved into place in every layer
        _commit("commit_small", 1, 5, 28, 8, 128, 16, 300),
        # a block's accepted rows of 64 requests moved into place in every layer
        _commit("commit_block", 64, 16, 32, 8, 128, 16, 256),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50.0)


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "logp", "logp", "grad", "commit"])
    if op == "attn":
        heads, kv = rng.choice([(32, 8), (16, 2), (32, 4), (16, 16), (28, 4), (12, 12), (64, 8), (8, 1), (40, 8)])
        dim = rng.choice([64, 64, 96, 128, 128, 128, 128, 256])
        kind = rng.choice(["decode", "chain", "ragged", "tree"])
        rows = 1 if kind == "decode" else _log_int(rng, 2, 16) if kind != "tree" else _log_int(rng, 3, 60)
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        batch = _log_int(rng, 1, 256)
        hi = _log_int(rng, 2, 100000)
        lo = rng.randint(0, hi)
        page = rng.choice([1, 16, 16, 32, 64, 5])
        staged = rng.random() < 0.4

        def case():
            return _attn(None, batch, rows, lo, hi, heads, kv, dim, page, dtype, kind == "ragged", kind == "tree", staged)

        most = _cost(_attn(None, 128, 1, 64, 8192, 32, 8, 128, 16)) * (1.0 if dtype == "bf16" else 0.5)
        while (_cost(case()) > most or batch * hi * kv * dim > 1 << 30  # the padded plain form has to fit too
               or batch * hi * heads * rows > 1 << 29):
            if batch > 1 and (hi < 64 or rng.random() < 0.5):
                batch = max(1, batch // 2)
            else:
                hi = max(1, hi // 2)
                lo = min(lo, hi)
        return case()
    if op == "commit":
        return _commit(None, _log_int(rng, 1, 64), _log_int(rng, 2, 16), rng.randint(1, 32), rng.choice([1, 2, 4, 8]),
                       rng.choice([64, 128, 256, 96]), rng.choice([1, 16, 32, 7]), rng.randint(1, 256),
                       rng.choice(["bf16", "bf16", "f32"]))
    vocab = rng.choice([32000, 128256, 151936, 32003, _log_int(rng, 500, 150000)])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    rows = min(_log_int(rng, 1, 1024), (1024 * 151936 * 2) // (vocab * (2 if dtype == "bf16" else 4)))
    if op == "logp":
        return _logp(None, rows, vocab, dtype, rng.randint(1, 4), rng.choice([0, 1, 5, 20, 20]), rng.random() < 0.5,
                     rng.choice([1.0, 0.4]), rng.choice([0, 0, 3]))
    return _grad(None, rows, vocab, dtype, rng.randint(1, 4), rng.choice([0, 0, 5]), rng.random() < 0.5,
                 rng.random() < 0.5)


# ----------------------------------------------------------------------------------------------------------------------
# What a case fixes: lengths, trees, accepted counts
# ----------------------------------------------------------------------------------------------------------------------


def _spread(i):
    return ((i + 1) * GOLDEN) % 1.0


def _lengths(case):
    """Committed tokens of each request, between lo and hi, and its new rows."""
    lens = [case["lo"] + int((case["hi"] - case["lo"]) * _spread(i) + 0.5) for i in range(case["batch"])]
    rows = [1 + int(case["rows"] * _spread(3 * i + 1)) if case["ragged"] else case["rows"] for i in range(case["batch"])]
    return lens, rows


def _parents(case, b):
    """A draft tree: mostly a chain of its last levels, some branching."""
    r = random.Random(7919 * b + case["rows"])
    return [-1] + [r.randint(max(0, i - 4), i - 1) for i in range(1, case["rows"])]


def _accepted(case):
    """Committed entries of each request (accepted drafts and the anchor)."""
    return [1 + int(case["rows"] * _spread(i) ** 2) for i in range(case["batch"])]


def _visible(case):
    """[batch, rows, rows] lists of what each new row sees among the new rows."""
    n = case["rows"]
    if not case["tree"]:
        return None
    out = []
    for b in range(case["batch"]):
        par, m = _parents(case, b), []
        for i in range(n):
            row = list(m[par[i]]) if i else [0] * n
            row[i] = 1
            m.append(row)
        out.append(m)
    return out


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "attn":
        lens, rows = _lengths(case)
        H, G, D = case["heads"], case["kv_heads"], case["head_dim"]
        vis = _visible(case)
        keys = sum(lens) + sum(rows)
        pairs = 0
        for b in range(case["batch"]):
            among = sum(map(sum, vis[b])) if vis else rows[b] * (rows[b] + 1) // 2
            pairs += rows[b] * lens[b] + among
        table = sum(-(-n // case["page"]) for n in lens) * 4
        return {"bytes": keys * G * D * 2 * es + sum(rows) * H * (2 * D * es + 4) + table, "flops": 4.0 * D * H * pairs}
    if case["op"] == "commit":
        n = sum(_accepted(case)) * case["layers"] * 2 * case["kv_heads"] * case["head_dim"] * es
        return {"bytes": 2 * n, "flops": 0}
    n = case["rows"]
    if case["op"] == "logp":
        live = _live(case)
        return {"bytes": live * case["vocab"] * es + n * (8 * case["ids"] + 8 * case["top"] + 20),
                "flops": 7.0 * live * case["vocab"]}
    return {"bytes": 2 * n * case["vocab"] * es + n * (8 * case["ids"] + 8 * case["top"] + 20),
            "flops": 7.0 * n * case["vocab"]}


def _live(case):
    return max(1, int(case["rows"] * case["live"]))


# ----------------------------------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------------------------------


def _padded(rows, cols, dtype):
    """A [rows, cols] view whose row stride is a multiple of 16 bytes."""
    per = 16 // dtype.itemsize
    return torch.zeros(rows, -(-cols // per) * per, dtype=dtype, device=DEV)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)
    return {"attn": _prepare_attn, "commit": _prepare_commit, "logp": _prepare_logp, "grad": _prepare_grad}[case["op"]](case, g)


def _pool(pages, page, kv_heads, head_dim, dtype, g, layers=1):
    shape = (layers, pages, page, kv_heads, head_dim)
    return [torch.randn(shape, generator=g, dtype=dtype, device=DEV) for _ in range(2)]


def _prepare_attn(case, g):
    B, n, page = case["batch"], case["rows"], case["page"]
    dt = DTYPES[case["dtype"]]
    lens, rows = _lengths(case)
    total = sum(rows)
    room = [L + (0 if case["staged"] else r) for L, r in zip(lens, rows)]  # drafts in place follow the history
    need = [max(1, -(-x // page)) for x in room]
    spare = -(-total // page) if case["staged"] else 0
    pages = sum(need) + spare
    k, v = _pool(pages, page, case["kv_heads"], case["head_dim"], dt, g)
    order = torch.randperm(pages, generator=g, device=DEV)
    table = torch.zeros(B, max(need), dtype=torch.int32, device=DEV)
    own_page = torch.arange(max(need), device=DEV)[None, :] < torch.tensor(need, device=DEV)[:, None]
    table[own_page] = order[:sum(need)].int()
    q = 2.0 * torch.randn(total, case["heads"], case["head_dim"], generator=g, device=DEV)
    s = {"case": case, "k": k, "v": v, "table": table, "q": q.to(dt), "scale": case["head_dim"] ** -0.5,
         "seq_lens": torch.tensor(lens, dtype=torch.int64, device=DEV), "max_len": n,
         "cu": None, "slots": None, "mask": None}
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    if case["ragged"]:
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    if case["staged"]:
        s["slots"] = (order[sum(need):][:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:total].contiguous()
    if case["tree"]:
        s["mask"] = torch.tensor(_visible(case), dtype=torch.uint8, device=DEV)
    if own:
        from reject_row_vocab_gb300 import specverify as sv
        s["cache"] = sv.PagedKvCache(k, v, table)
        s["out"] = sv.AttentionOutputs.allocate(total, case["heads"], case["head_dim"], B, dt)
        s["ws"] = sv.attention_workspace(B, n, s["cache"], case["heads"])
    return s


def _prepare_commit(case, g):
    B, n, page = case["batch"], case["rows"], case["page"]
    dt = DTYPES[case["dtype"]]
    acc = _accepted(case)
    need = -(-(case["length"] + n + 1) // page)
    spare = -(-B * n // page)
    k, v = _pool(B * need + spare, page, case["kv_heads"], case["head_dim"], dt, g, case["layers"])
    order = torch.randperm(B * need + spare, generator=g, device=DEV)
    table = order[:B * need].reshape(B, need).int().contiguous()
    slots = (order[B * need:][:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:B * n]
    cu = [0]
    for a in acc:
        cu.append(cu[-1] + a)
    # an accepted path: the anchor's row, then rows further on in rising order
    prio = torch.rand(B, n, generator=g, device=DEV)
    prio[:, 0] = 2.0
    rank = prio.argsort(1, descending=True).argsort(1)
    keep = rank < torch.tensor([min(a, n) for a in acc], device=DEV)[:, None]
    src = slots.reshape(B, n)[keep]
    start = torch.full((B,), case["length"], dtype=torch.int64, device=DEV)
    within = torch.arange(cu[-1], device=DEV) - torch.repeat_interleave(torch.tensor(cu[:-1], device=DEV),
                                                                         torch.tensor(acc, device=DEV))
    dst = torch.repeat_interleave(start, torch.tensor(acc, device=DEV)) + within
    pad = B * n - cu[-1]
    s = {"case": case, "k": k, "v": v, "table": table, "cu": torch.tensor(cu, dtype=torch.int32, device=DEV),
         "src": torch.cat([src, torch.full((pad,), -1, dtype=torch.int64, device=DEV)]),
         "dst": torch.cat([dst, torch.full((pad,), -1, dtype=torch.int64, device=DEV)]), "max_len": n}
    if own:
        from reject_row_vocab_gb300 import specverify as sv
        s["cache"] = sv.PagedKvCache(k, v, table)
        s["status"] = torch.empty(B, dtype=torch.int32, device=DEV)
    return s


def _logits(case, g, rows, masked=0):
    """N(0, 3^2) logits with one likely token a row; `masked` of 8 rows keep a grammar's few tokens only."""
    V = case["vocab"]
    x = 3.0 * torch.randn(rows, V, generator=g, device=DEV)
    hot = torch.randint(0, V, (rows, 1), generator=g, device=DEV)
    x.scatter_add_(1, hot, torch.full((rows, 1), 6.0, device=DEV))
    if masked:
        drop = torch.rand(rows, V, generator=g, device=DEV) > 0.01
        drop &= (torch.arange(rows, device=DEV) % 8 < masked)[:, None]
        drop.scatter_(1, hot, False)
        x.masked_fill_(drop, float("-inf"))
    out = _padded(rows, V, DTYPES[case["dtype"]])
    out.copy_(x)
    return out, hot


def _given(case, g, rows, hot):
    ids = torch.randint(0, case["vocab"], (rows, case["ids"]), generator=g, device=DEV)
    likely = torch.rand(rows, generator=g, device=DEV) < 0.7
    ids[:, 0] = torch.where(likely, hot[:, 0], ids[:, 0])
    return ids.int()


def _temps(case, g, rows):
    if not case["temp"]:
        return None
    t = 0.5 + 0.7 * torch.rand(rows, generator=g, device=DEV)
    t[::5] = 0.0  # greedy requests report the unscaled distribution
    return t


def _prepare_logp(case, g):
    n, live = case["rows"], _live(case)
    logits, hot = _logits(case, g, n, case["masked"])
    s = {"case": case, "logits": logits, "temp": _temps(case, g, n), "index": None, "ids": _given(case, g, n, hot)}
    if case["live"] < 1.0:  # the committed rows of a verify call, padded with -1
        pick = torch.randperm(n, generator=g, device=DEV)[:live].sort().values
        at = torch.randperm(n, generator=g, device=DEV)[:live].sort().values
        s["index"] = torch.full((n,), -1, dtype=torch.int32, device=DEV)
        s["index"][at] = pick.int()
        ids = torch.full_like(s["ids"], -1)
        ids[at] = s["ids"][pick]
        s["ids"] = ids
    if own:
        from reject_row_vocab_gb300 import specverify as sv
        s["out"] = sv.LogprobOutputs.allocate(n, case["ids"], case["top"])
        s["ws"] = sv.logprobs_workspace(n, case["vocab"], case["top"])
    return s


def _prepare_grad(case, g):
    n = case["rows"]
    logits, hot = _logits(case, g, n)
    s = {"case": case, "logits": logits, "temp": _temps(case, g, n), "ids": _given(case, g, n, hot)}
    # what the forward pass kept: the rows' maxima, log sums and entropies, and the alternatives
    l = logits.double()
    T = _scale(s["temp"], n).double()[:, None]
    s["max"] = l.amax(1)
    e = torch.exp((l - s["max"][:, None]) / T)
    z = e.sum(1)
    s["entropy"] = (z.log() - (e * ((l - s["max"][:, None]) / T)).sum(1) / z).float()
    s["logz"], s["max"] = z.log().float(), s["max"].float()
    s["top_ids"] = l.sort(dim=1, descending=True, stable=True).indices[:, :case["top"]].int().contiguous() if case["top"] else None
    s["g_lp"] = -torch.rand(n, case["ids"], generator=g, device=DEV)
    s["g_top"] = 0.2 * torch.randn(n, case["top"], generator=g, device=DEV) if case["top"] else None
    s["g_ent"] = 0.01 * torch.randn(n, generator=g, device=DEV) if case["entropy"] else None
    if own:
        from reject_row_vocab_gb300 import specverify as sv
        s["kept"] = sv.LogprobOutputs(logprob=None, entropy=s["entropy"], row_max=s["max"], log_z=s["logz"],
                                      top_ids=s["top_ids"], top_logprob=None, flags=None)
        s["out"] = torch.empty_like(logits.as_strided((n, logits.stride(0)), logits.stride()))[:, :case["vocab"]]
    return s


# ----------------------------------------------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"attn": _plain_attn, "commit": _plain_commit, "logp": _plain_logp, "grad": _plain_grad}[op](s)
    from reject_row_vocab_gb300 import specverify as sv
    if op == "attn":
        o = sv.paged_attention(s["q"], s["cache"], s["seq_lens"], max_len=s["max_len"], cu_seqlens=s["cu"],
                               row_slots=s["slots"], mask=s["mask"], scale=s["scale"], out=s["out"], ws=s["ws"])
        return {"out": o.out, "lse": o.lse}
    if op == "commit":
        sv.kv_commit(s["cache"], s["cu"], s["src"], s["dst"], max_len=s["max_len"], dev_status=s["status"])
        return {"k": s["k"], "v": s["v"]}
    if op == "logp":
        o = sv.token_logprobs(s["logits"], s["ids"], top_k=s["case"]["top"], row_index=s["index"], row_temp=s["temp"],
                              out=s["out"], ws=s["ws"])
        r = {"logprob": o.logprob, "entropy": o.entropy, "row_max": o.row_max, "log_z": o.log_z}
        return dict(r, top_ids=o.top_ids, top_logprob=o.top_logprob) if s["case"]["top"] else r
    return {"dlogits": sv.token_logprobs_backward(s["logits"], s["ids"], s["kept"], s["g_lp"], g_entropy=s["g_ent"],
                                                  g_top=s["g_top"], row_temp=s["temp"], out=s["out"])}


def _rows_of(s, B, n):
    """The global row of each request's i-th new row, and which of them there are."""
    i = torch.arange(n, device=DEV)
    if s["cu"] is None:
        return torch.arange(B, device=DEV)[:, None] * n + i, torch.ones(B, n, dtype=torch.bool, device=DEV)
    cu = s["cu"].long()
    have = i < (cu[1:] - cu[:-1])[:, None]
    return torch.where(have, cu[:-1, None] + i, 0), have


def _slot_of(table, pos, page):
    at = (pos // page).clamp(0, table.shape[1] - 1)
    return table.long().gather(1, at) * page + pos % page


def _plain_attn(s):
    c = s["case"]
    B, n, page, H, G, D = c["batch"], s["max_len"], c["page"], c["heads"], c["kv_heads"], c["head_dim"]
    lens = s["seq_lens"]
    row, have = _rows_of(s, B, n)
    P = c["hi"]
    pos = torch.arange(P, device=DEV).expand(B, P)
    i = torch.arange(n, device=DEV)
    new = s["slots"][row] if s["slots"] is not None else _slot_of(s["table"], lens[:, None] + i, page)
    slot = torch.cat([_slot_of(s["table"], pos, page), new], 1)
    among = s["mask"].bool() if s["mask"] is not None else (i[None, :] <= i[:, None]).expand(B, n, n)
    see = torch.cat([(pos < lens[:, None])[:, None, :].expand(B, n, P), among & have[:, None, :]], 2)
    there = torch.cat([pos < lens[:, None], have], 1)
    k = s["k"][0].reshape(-1, G, D)[torch.where(there, slot, 0)].float().permute(0, 2, 3, 1)
    v = s["v"][0].reshape(-1, G, D)[torch.where(there, slot, 0)].float().permute(0, 2, 1, 3)
    q = s["q"][row].float().reshape(B, n, G, H // G, D).permute(0, 2, 1, 3, 4).reshape(B, G, n * (H // G), D)
    x = (q @ k) * s["scale"]
    x = x.reshape(B, G, n, H // G, P + n).masked_fill(~see[:, None, :, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == float("-inf"), 0.0, m))
    z = e.sum(-1, keepdim=True)
    o = (e.reshape(B, G, n * (H // G), P + n) @ v).reshape(B, G, n, H // G, D) / torch.where(z == 0, 1.0, z)
    lse = (m + z.log())[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, n, H, D)
    lse = lse.permute(0, 2, 1, 3).reshape(B, n, H)
    return {"out": o[have].to(s["q"].dtype), "lse": lse[have]}


def _plain_commit(s):
    c = s["case"]
    page, total = c["page"], s["cu"][-1:]
    n = s["src"].numel()
    at = torch.arange(n, device=DEV)
    b = (torch.searchsorted(s["cu"], at.int(), right=True) - 1).clamp(0, c["batch"] - 1)
    live = at < total
    pos = torch.where(live, s["dst"], 0)
    dst = s["table"].long()[b, pos // page] * page + pos % page
    src = s["src"][live]
    dst = dst[live]
    for_k, for_v = (t.reshape(c["layers"], -1, c["kv_heads"], c["head_dim"]) for t in (s["k"], s["v"]))
    for_k[:, dst] = for_k[:, src]
    for_v[:, dst] = for_v[:, src]
    return {"k": s["k"], "v": s["v"]}


def _scale(temp, n):
    if temp is None:
        return torch.ones(n, device=DEV)
    return torch.where((temp >= 1e-30) & (temp < float("inf")), temp, 1.0)


def _plain_logp(s):
    c = s["case"]
    n, K, V = c["rows"], c["top"], c["vocab"]
    live = torch.ones(n, dtype=torch.bool, device=DEV) if s["index"] is None else s["index"] >= 0
    l = s["logits"].float() if s["index"] is None else s["logits"][s["index"].long()[live]].float()
    T = _scale(s["temp"], n)[live][:, None]
    m = l.amax(1, keepdim=True)
    d = (l - m) / T
    e = torch.exp(d)
    z = e.sum(1)
    h = z.log() - (e * torch.where(e > 0, d, 0.0)).sum(1) / z
    ids = s["ids"][live].long()
    lp = (l.gather(1, ids) - m) / T - z.log()[:, None]
    out = {"logprob": torch.zeros(n, c["ids"], device=DEV), "entropy": torch.zeros(n, device=DEV),
           "row_max": torch.full((n,), float("-inf"), device=DEV), "log_z": torch.zeros(n, device=DEV)}
    out["logprob"][live], out["entropy"][live], out["row_max"][live], out["log_z"][live] = lp, h, m[:, 0], z.log()
    if K:
        # rank by value (-0 as 0), then by the lower index: both in one whole number
        bits = (l + 0.0).view(torch.int32)
        key = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long() * (1 << 32) - torch.arange(V, device=DEV)
        top = key.topk(K, 1).indices
        val = l.gather(1, top)
        out["top_ids"] = torch.full((n, K), -1, dtype=torch.int32, device=DEV)
        out["top_logprob"] = torch.full((n, K), float("-inf"), device=DEV)
        out["top_ids"][live] = torch.where(val > float("-inf"), top, -1).int()
        out["top_logprob"][live] = (val - m) / T - z.log()[:, None]
    return out


def _plain_grad(s):
    c = s["case"]
    l = s["logits"].float()
    T = _scale(s["temp"], c["rows"])[:, None]
    lp = (l - s["max"][:, None]) / T - s["logz"][:, None]
    p = torch.exp(lp)
    G = s["g_lp"].sum(1, keepdim=True)
    if s["g_top"] is not None:
        G = G + s["g_top"].sum(1, keepdim=True)
    d = -p * G
    if s["g_ent"] is not None:
        d = d - s["g_ent"][:, None] * p * (lp + s["entropy"][:, None])
    d.scatter_add_(1, s["ids"].long(), s["g_lp"])
    if s["g_top"] is not None:
        d.scatter_add_(1, s["top_ids"].long(), s["g_top"])
    return {"dlogits": (d / T).to(s["logits"].dtype)}


# ----------------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits, request by request and row by row
# ----------------------------------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "commit": _exact_commit, "logp": _exact_logp, "grad": _exact_grad}[case["op"]](s)


def _exact_attn(s):
    c = s["case"]
    lens, rows = _lengths(c)
    page, H, G, D = c["page"], c["heads"], c["kv_heads"], c["head_dim"]
    kf, vf = s["k"].reshape(-1, G, D), s["v"].reshape(-1, G, D)
    outs, lses, at = [], [], 0
    for b in range(c["batch"]):
        L, r = lens[b], rows[b]
        table = s["table"][b].long()
        pos = torch.arange(L + (0 if c["staged"] else r), device=DEV)
        slot = table[torch.div(pos, page, rounding_mode="floor")] * page + torch.remainder(pos, page)
        if c["staged"]:
            slot = torch.cat([slot, s["slots"][at:at + r]])
        k, v = kf[slot].double(), vf[slot].double()
        q = s["q"][at:at + r].double()
        see = torch.ones(r, L + r, dtype=torch.bool, device=DEV)
        see[:, L:] = s["mask"][b, :r, :r].bool() if s["mask"] is not None else torch.ones(r, r, device=DEV).tril().bool()
        o, z = torch.empty(r, H, D, dtype=torch.float64, device=DEV), torch.empty(r, H, dtype=torch.float64, device=DEV)
        for h in range(G):
            mine = slice(h * (H // G), (h + 1) * (H // G))
            x = torch.einsum("rgd,kd->rgk", q[:, mine], k[:, h]) * s["scale"]
            x = torch.where(see[:, None, :], x, float("-inf"))
            z[:, mine] = torch.logsumexp(x, -1)
            o[:, mine] = torch.einsum("rgk,kd->rgd", torch.softmax(x, -1), v[:, h])
        outs.append(o)
        lses.append(z)
        at += r
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_commit(s):
    c = s["case"]
    cu, src, dst, table = s["cu"].tolist(), s["src"].tolist(), s["dst"].tolist(), s["table"].tolist()
    page = c["page"]
    k, v = s["k"].double(), s["v"].double()
    k0, v0 = s["k"], s["v"]
    for b in range(c["batch"]):
        for j in range(cu[b], cu[b + 1]):
            to, off = table[b][dst[j] // page], dst[j] % page
            k[:, to, off] = k0[:, src[j] // page, src[j] % page].double()
            v[:, to, off] = v0[:, src[j] // page, src[j] % page].double()
    return {"k": k, "v": v}


def _exact_logp(s):
    c = s["case"]
    n, K = c["rows"], c["top"]
    f64 = dict(dtype=torch.float64, device=DEV)
    out = {"logprob": torch.zeros(n, c["ids"], **f64), "entropy": torch.zeros(n, **f64),
           "row_max": torch.full((n,), float("-inf"), **f64), "log_z": torch.zeros(n, **f64)}
    if K:
        out["top_ids"] = None
        out["top_logprob"] = torch.full((n, K), float("-inf"), **f64)
    index = list(range(n)) if s["index"] is None else s["index"].tolist()
    temp = [1.0] * n if s["temp"] is None else s["temp"].tolist()
    for i, r in enumerate(index):
        if r < 0:
            continue
        T = torch.tensor(temp[i] if 1e-30 <= temp[i] < math.inf else 1.0, dtype=torch.float64, device=DEV)
        l = s["logits"][r].double()
        lp = torch.log_softmax(l / T, 0)
        p = lp.exp()
        out["logprob"][i] = lp[s["ids"][i].long()]
        out["entropy"][i] = -torch.where(p > 0, p * lp, 0.0).sum()
        out["row_max"][i] = l.max()
        out["log_z"][i] = torch.logsumexp((l - l.max()) / T, 0)
        if K:
            out["top_logprob"][i] = lp.sort(descending=True).values[:K]
    return out


def _exact_grad(s):
    c = s["case"]
    l = s["logits"].double().requires_grad_(True)
    T = _scale(s["temp"], c["rows"]).double()[:, None]
    with torch.enable_grad():
        lp = torch.log_softmax(l / T, 1)
        loss = (lp.gather(1, s["ids"].long()) * s["g_lp"].double()).sum()
        if s["g_top"] is not None:
            loss = loss + (lp.gather(1, s["top_ids"].long()) * s["g_top"].double()).sum()
        if s["g_ent"] is not None:
            loss = loss + (-(lp.exp() * lp).sum(1) * s["g_ent"].double()).sum()
        return {"dlogits": torch.autograd.grad(loss, l)[0]}
