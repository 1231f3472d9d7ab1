"""What the operators that fill and read a KV cache are measured on: appending rotated keys and values to a paged cache in
bf16 or fp32 and to one held in 4 bits, and attention, the commit's move and reading back in the 4-bit cache.

`run` computes each operator in its plain form (elementary torch operations), or, where `own` is true, through the
library's public entry points.  Lengths, trees and accepted counts are functions of the case alone, so that `work` can count
them; values come from the seed.

The 4-bit format: the values of 16 neighbouring columns share a scale; a value is the scale times a code.  Codes have a sign
and three bits for 0, 0.5, 1, 1.5, 2, 3, 4, 6 (two a byte, the even column in the lower half); a scale is a byte with five
exponent and three mantissa bits, the upper half of a positive half float without its sign bit, at most 10240.  The block of a
page and head holds K's codes, V's codes, K's scales and V's scales, up to a multiple of 16 bytes.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GOLDEN = 0.6180339887498949
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GROUP = 16
MOST = 10240.0  # the largest scale


# ----------------------------------------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------------------------------------


def _append(name, batch, rows, lo, hi, heads, kv_heads, head_dim, page, dtype="bf16", packed=False, ragged=False,
            tree=False, pairs=0, interleaved=False, far=0):
    """rows: new rows a request (ragged: up to that); pairs: rotated pairs of columns (0: all); tree: positions by depth and
    places given as slots; far: what is added to a tree's positions."""
    c = {"op": "append", "batch": batch, "rows": rows, "lo": lo, "hi": hi, "heads": heads, "kv_heads": kv_heads,
         "head_dim": head_dim, "page": page, "dtype": dtype, "packed": packed, "ragged": ragged, "tree": tree,
         "pairs": pairs or head_dim // 2, "interleaved": interleaved, "far": far}
    return dict(c, name=name) if name else c


def _attn(name, batch, rows, lo, hi, heads, kv_heads, head_dim, page, ragged=False, tree=False, staged=False):
    c = {"op": "attn", "batch": batch, "rows": rows, "lo": lo, "hi": hi, "heads": heads, "kv_heads": kv_heads,
         "head_dim": head_dim, "page": page, "dtype": "bf16", "packed": True, "ragged": ragged, "tree": tree,
         "staged": staged}
    return dict(c, name=name) if name else c


def _commit(name, batch, rows, layers, kv_heads, head_dim, page, length):
    c = {"op": "commit", "batch": batch, "rows": rows, "layers": layers, "kv_heads": kv_heads, "head_dim": head_dim,
         "page": page, "length": length, "dtype": "bf16", "packed": True}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one layer's call of one request decoding a token: its query is rotated, its key and value go into the cache
        _append("append_token", 1, 1, 500, 500, 32, 8, 128, 16),
        # a prefill step of 12 requests, chunks of 1 to 1365 new tokens each behind what they have already
        _append("append_chunk", 12, 1365, 0, 4000, 32, 8, 128, 16, ragged=True),
        # a small fp32 model, draft trees far along in a long document, half of a head's columns rotated in neighbouring pairs,
        # the rows staged in a pool of single slots
        _append("append_tree_f32", 16, 17, 37, 2100, 8, 4, 64, 1, dtype="f32", tree=True, pairs=16, interleaved=True,
                far=1000000),
        # a full decoding batch's tokens into the 4-bit cache, and the rows read back as the values that it now holds
        _append("packed_append_batch", 256, 1, 64, 2000, 32, 8, 128, 16, packed=True),
        # a prefill step into the 4-bit cache, read back
        _append("packed_append_chunk", 12, 1365, 0, 4000, 32, 8, 128, 16, packed=True, ragged=True),
        # one request's accepted chain moved into place in every layer of the 4-bit cache, and read back
        _commit("packed_commit_small", 1, 5, 28, 8, 128, 16, 300),
        # a block's accepted rows of 64 requests
        _commit("packed_commit_block", 64, 16, 32, 8, 128, 16, 256),
        # one request decoding one token over a short history: a chat's first answer, where latency counts
        _attn("packed_attn_token", 1, 1, 500, 500, 32, 8, 128, 16),
        # a full decoding batch with histories of very different lengths, one token each
        _attn("packed_attn_batch", 128, 1, 64, 8192, 32, 8, 128, 16),
        # a 64-request block of 16 rows (anchor and 15 drafts) a request, drafts in place behind the history
        _attn("packed_attn_block", 64, 16, 100, 4000, 32, 8, 128, 64),
        # 16 requests' draft trees of 17 nodes, a pool of single slots, the drafts staged elsewhere in the pool
        _attn("packed_attn_tree", 16, 17, 37, 2100, 16, 2, 128, 1, tree=True, staged=True),
        # two requests of a long document, 5 rows each: few rows, so the length is split over the whole GPU
        _attn("packed_attn_long", 2, 5, 60000, 100000, 32, 4, 128, 32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 100.0)


def draw(rng):
    op = rng.choice(["append", "append", "append", "attn", "attn", "attn", "commit"])
    page = rng.choice([1, 16, 16, 32, 64, 5])
    if op == "commit":
        return _commit(None, _log_int(rng, 1, 64), _log_int(rng, 2, 16), rng.randint(1, 32), rng.choice([1, 2, 4, 8]),
                       rng.choice([64, 128, 256, 96]), page, rng.randint(1, 256))
    heads, kv = rng.choice([(32, 8), (16, 2), (32, 4), (16, 16), (28, 4), (12, 12), (64, 8), (8, 1), (40, 8)])
    dim = rng.choice([64, 64, 96, 128, 128, 128, 128, 256])
    if op == "append":
        packed = rng.random() < 0.6
        kind = rng.choice(["decode", "chunk", "chunk", "tree"])
        batch = _log_int(rng, 1, 256)
        rows = 1 if kind == "decode" else _log_int(rng, 2, 4000) if kind == "chunk" else _log_int(rng, 3, 60)
        hi = _log_int(rng, 2, 4000)
        lo = rng.randint(0, hi)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        pairs = rng.choice([dim // 2, dim // 2, dim // 4, rng.randint(1, dim // 2)])
        inter = rng.random() < 0.4
        far = rng.choice([0, 0, _log_int(rng, 1000, 4000000)]) if kind == "tree" else 0

        def case():
            return _append(None, batch, rows, lo, hi, heads, kv, dim, page, dtype, packed, kind == "chunk", kind == "tree",
                           pairs, inter, far)

        most = _cost(_append(None, 12, 1365, 0, 4000, 32, 8, 128, 16, packed=True, ragged=True))
        while _cost(case()) > most or batch * (hi + rows) * kv * dim > 1 << 28:
            if batch > 1 and (rows < 8 or rng.random() < 0.5):
                batch = max(1, batch // 2)
            elif rows > 8 and rng.random() < 0.6:
                rows = rows // 2
            else:
                hi = max(1, hi // 2)
                lo = min(lo, hi)
        return case()
    kind = rng.choice(["decode", "chain", "ragged", "tree"])
    rows = 1 if kind == "decode" else _log_int(rng, 2, 16) if kind != "tree" else _log_int(rng, 3, 60)
    batch = _log_int(rng, 1, 256)
    hi = _log_int(rng, 2, 100000)
    lo = rng.randint(0, hi)
    staged = rng.random() < 0.4

    def case():
        return _attn(None, batch, rows, lo, hi, heads, kv, dim, page, kind == "ragged", kind == "tree", staged)

    most = _cost(_attn(None, 128, 1, 64, 8192, 32, 8, 128, 16))
    while (_cost(case()) > most or batch * hi * kv * dim > 1 << 30  # the padded plain form has to fit too
           or batch * hi * heads * rows > 1 << 29):
        if batch > 1 and (hi < 64 or rng.random() < 0.5):
            batch = max(1, batch // 2)
        else:
            hi = max(1, hi // 2)
            lo = min(lo, hi)
    return case()


# ----------------------------------------------------------------------------------------------------------------------
# What a case fixes: lengths, trees, accepted counts
# ----------------------------------------------------------------------------------------------------------------------


def _spread(i):
    return ((i + 1) * GOLDEN) % 1.0


def _lengths(case):
    """Committed tokens of each request, between lo and hi, and its new rows."""
    lens = [case["lo"] + int((case["hi"] - case["lo"]) * _spread(i) + 0.5) for i in range(case["batch"])]
    rows = [min(case["rows"], 1 + int(case["rows"] * _spread(3 * i + 1))) if case["ragged"] else case["rows"]
            for i in range(case["batch"])]
    return lens, rows


def _parents(case, b):
    """A draft tree: mostly a chain of its last levels, some branching."""
    r = random.Random(7919 * b + case["rows"])
    return [-1] + [r.randint(max(0, i - 4), i - 1) for i in range(1, case["rows"])]


def _depths(case, b):
    d = []
    for p in _parents(case, b):
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _accepted(case):
    """Committed entries of each request (accepted drafts and the anchor)."""
    return [min(case["rows"], 1 + int(case["rows"] * _spread(i) ** 2)) for i in range(case["batch"])]


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


def _block_bytes(page, dim):
    return (page * dim * 9 // 8 + 15) // 16 * 16


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    G, D = case["kv_heads"], case["head_dim"]
    entry = 2 * G * D  # values of K and V of a row
    if case["op"] == "append":
        lens, rows = _lengths(case)
        n, H = sum(rows), case["heads"]
        small = n * (16 if case["tree"] else 4) + case["batch"] * 8 + case["pairs"] * 4
        held = n * entry * 9 // 16 if case["packed"] else n * entry * es
        back = n * entry * 9 // 16 + n * entry * es if case["packed"] else 0
        return {"bytes": n * (H * D + entry) * es + n * H * D * es + held + back + small,
                "flops": 6.0 * n * (H + G) * case["pairs"] + (8.0 * n * entry if case["packed"] else 0.0)}
    if case["op"] == "commit":
        n = sum(_accepted(case)) * case["layers"] * entry
        return {"bytes": 2 * (n * 9 // 16) + n * 9 // 16 + n * es, "flops": float(n)}
    lens, rows = _lengths(case)
    H = case["heads"]
    vis = _visible(case)
    keys = sum(lens) + sum(rows)
    pairs = 0
    for b in range(case["batch"]):
        among = sum(map(sum, vis[b])) if vis else rows[b] * (rows[b] + 1) // 2
        pairs += rows[b] * lens[b] + among
    table = sum(-(-n // case["page"]) for n in lens) * 4
    return {"bytes": keys * entry * 9 // 16 + sum(rows) * H * (2 * D * es + 4) + table, "flops": 4.0 * D * H * pairs}


# ----------------------------------------------------------------------------------------------------------------------
# The 4-bit format in plain operations
# ----------------------------------------------------------------------------------------------------------------------


def _quantize(x):
    """Codes (as bytes of 0..15) and scales (as bytes) of x [..., dim], and the values that they stand for."""
    y = x.unflatten(-1, (-1, GROUP))
    top = y.abs().amax(-1, keepdim=True)
    e = torch.frexp((top / 6.0).clamp(2.0 ** -14, MOST)).exponent - 4
    step = torch.tensor([2.0 ** i for i in range(-17, 11)], dtype=x.dtype, device=x.device)[e + 17]
    s = (torch.round(top / (6.0 * step)) * step).clamp(max=MOST)  # (half way between two scales: only this quotient is exact)
    a = y.abs()
    code = torch.zeros_like(y, dtype=torch.uint8)
    for i in range(7):  # a value between two codes goes to the nearer one, half way to the even one
        half = s * ((CODES[i] + CODES[i + 1]) / 2)
        code += (a > half) | ((a == half) & (i % 2 == 1) & (half > 0))
    scale = (s.to(torch.float16).view(torch.int16) >> 7).to(torch.uint8)[..., 0]
    mag = torch.tensor(CODES, dtype=x.dtype, device=x.device)[code.int()]
    value = torch.where(y < 0, -mag, mag) * s
    code = code | ((y < 0).to(torch.uint8) << 3)
    return code.flatten(-2), scale, value.flatten(-2)


def _parts(data, page, dim):
    """Views of a packed cache [layers, pages, heads, block]: K's and V's codes and scales, [layers, pages, heads, page, .]."""
    c, s = page * dim // 2, page * dim // 16
    cut = lambda at, n, cols: data[..., at:at + n].unflatten(-1, (page, cols))
    return cut(0, c, dim // 2), cut(c, c, dim // 2), cut(2 * c, s, dim // 16), cut(2 * c + s, s, dim // 16)


def _values(codes, scales, dtype=torch.float32):
    """The values of packed codes [..., dim / 2] and scales [..., dim / 16]."""
    table = torch.tensor([s * m for s in (1.0, -1.0) for m in CODES], dtype=dtype, device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    s = (scales.to(torch.int16) << 7).view(torch.float16).to(dtype)
    return (v.unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


def _packed_pool(layers, pages, page, heads, dim, g):
    """A packed cache of normal values, quantised piece by piece."""
    data = torch.zeros(layers, pages, heads, _block_bytes(page, dim), dtype=torch.uint8, device=DEV)
    parts = _parts(data.flatten(0, 1)[None], page, dim)
    step = max(1, (1 << 25) // (heads * page * dim))
    for i in range(0, layers * pages, step):
        n = min(step, layers * pages - i)
        for j in range(2):
            x = torch.randn(n, heads, page, dim, generator=g, device=DEV)
            y = x.unflatten(-1, (-1, GROUP))
            s = (y.abs().amax(-1, keepdim=True) / 6.0).to(torch.float16)
            byte = ((s.view(torch.int16) + 64) >> 7)  # to the nearest: the inputs need no ties
            s = (byte << 7).view(torch.float16).float()
            a = (y / s).abs()
            code = torch.bucketize(a, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV), out_int32=True)
            code = (code + 8 * (y < 0)).to(torch.uint8).flatten(-2)
            parts[j][0, i:i + n] = code[..., 0::2] | (code[..., 1::2] << 4)
            parts[2 + j][0, i:i + n] = byte[..., 0].to(torch.uint8)
    return data


# ----------------------------------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 29)
    return {"append": _prepare_append, "attn": _prepare_attn, "commit": _prepare_commit}[case["op"]](case, g)


def _table(case, lens, rows, staged, g):
    """Pages in random order: [batch, pages] and the slots of the staged rows."""
    B, page = case["batch"], case["page"]
    need = [max(1, -(-(L + (0 if staged else r)) // page)) for L, r in zip(lens, rows)]  # rows in place follow the history
    total = sum(rows)
    spare = -(-total // page) if staged else 0
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g, device=DEV)
    table = torch.zeros(B, max(need), dtype=torch.int32, device=DEV)
    table[torch.arange(max(need), device=DEV)[None, :] < torch.tensor(need, device=DEV)[:, None]] = order[:sum(need)].int()
    slots = None
    if staged:
        slots = (order[sum(need):][:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:total].contiguous()
    return pages, table, slots


def _cu(rows):
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _own_cache(s, k=None, v=None):
    from reject_row_vocab_gb300 import specverify as sv
    c = s["case"]
    if c["packed"]:
        return sv.PackedKvCache(s["data"], s["table"], page_size=c["page"], head_dim=c["head_dim"], dtype=DTYPES[c["dtype"]])
    return sv.PagedKvCache(k, v, s["table"])


def _prepare_append(case, g):
    B, page, H, G, D = case["batch"], case["page"], case["heads"], case["kv_heads"], case["head_dim"]
    dt = DTYPES[case["dtype"]]
    lens, rows = _lengths(case)
    total = sum(rows)
    pages, table, slots = _table(case, lens, rows, case["tree"], g)
    qkv = torch.randn(total, H + 2 * G, D, generator=g, device=DEV)
    # some columns of keys are large in every row, as in real models
    qkv[:, H:H + G] *= torch.where(torch.rand(G, D, generator=g, device=DEV) < 0.03, 8.0, 1.0)
    qkv = qkv.to(dt)
    n = case["pairs"]
    s = {"case": case, "table": table, "slots": slots, "qkv": qkv, "q": qkv[:, :H], "knew": qkv[:, H:H + G],
         "vnew": qkv[:, H + G:], "seq_lens": torch.tensor(lens, dtype=torch.int64, device=DEV), "max_len": max(rows),
         "cu": _cu(rows) if case["ragged"] else None, "positions": None, "rows": rows,
         "inv_freq": (10000.0 ** (-torch.arange(n, dtype=torch.float64, device=DEV) / n)).float()}
    if case["tree"]:
        s["positions"] = torch.tensor([lens[b] + case["far"] + d for b in range(B) for d in _depths(case, b)],
                                      dtype=torch.int64, device=DEV)
    if case["packed"]:
        s["data"] = _packed_pool(1, pages, page, G, D, g)
    else:
        s["k"], s["v"] = [torch.randn(1, pages, page, G, D, generator=g, dtype=dt, device=DEV) for _ in range(2)]
    if own:
        from reject_row_vocab_gb300 import specverify as sv
        s["cache"] = _own_cache(s, s.get("k"), s.get("v"))
        s["rotation"] = sv.Rotation(s["inv_freq"], interleaved=case["interleaved"])
        s["out"] = sv.KvAppendOutputs.allocate(total, H, D, B, dt)
        if case["packed"]:
            s["read"] = sv.KvReadOutputs.allocate(total, G, D, B, dt)
    return s


def _prepare_attn(case, g):
    lens, rows = _lengths(case)
    total = sum(rows)
    pages, table, slots = _table(case, lens, rows, case["staged"], g)
    q = 2.0 * torch.randn(total, case["heads"], case["head_dim"], generator=g, device=DEV)
    s = {"case": case, "table": table, "slots": slots, "q": q.bfloat16(), "scale": case["head_dim"] ** -0.5,
         "seq_lens": torch.tensor(lens, dtype=torch.int64, device=DEV), "max_len": max(rows),
         "cu": _cu(rows) if case["ragged"] else None, "mask": None,
         "data": _packed_pool(1, pages, case["page"], case["kv_heads"], case["head_dim"], g)}
    if case["tree"]:
        s["mask"] = torch.tensor(_visible(case), dtype=torch.uint8, device=DEV)
    if own:
        from reject_row_vocab_gb300 import specverify as sv
        s["cache"] = _own_cache(s)
        s["out"] = sv.AttentionOutputs.allocate(total, case["heads"], case["head_dim"], case["batch"], torch.bfloat16)
        s["ws"] = sv.attention_workspace(case["batch"], s["max_len"], s["cache"], case["heads"])
    return s


def _prepare_commit(case, g):
    B, n, page = case["batch"], case["rows"], case["page"]
    acc = _accepted(case)
    total = sum(acc)
    need = -(-(case["length"] + n + 1) // page)
    spare = -(-B * n // page)
    order = torch.randperm(B * need + spare, generator=g, device=DEV)
    table = order[:B * need].reshape(B, need).int().contiguous()
    slots = (order[B * need:][:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:B * n].reshape(B, n)
    # an accepted path: the anchor's row, then rows further on in rising order
    prio = torch.rand(B, n, generator=g, device=DEV)
    prio[:, 0] = 2.0
    rank = prio.argsort(1, descending=True).argsort(1)
    src = slots[rank < torch.tensor(acc, device=DEV)[:, None]]
    cu = _cu(acc)
    within = torch.arange(total, device=DEV) - torch.repeat_interleave(cu[:-1].long(), torch.tensor(acc, device=DEV))
    pad = torch.full((B * n - total,), -1, dtype=torch.int64, device=DEV)
    s = {"case": case, "table": table, "cu": cu, "src": torch.cat([src, pad]),
         "dst": torch.cat([case["length"] + within, pad]), "total": total,
         "seq_lens": torch.full((B,), case["length"], dtype=torch.int64, device=DEV), "max_len": n,
         "data": _packed_pool(case["layers"], B * need + spare, page, case["kv_heads"], case["head_dim"], g)}
    if own:
        from reject_row_vocab_gb300 import specverify as sv
        s["cache"] = _own_cache(s)
        s["status"] = torch.empty(B, dtype=torch.int32, device=DEV)
        s["read"] = sv.KvReadOutputs.allocate(total, case["kv_heads"], case["head_dim"], B, torch.bfloat16,
                                              layers=case["layers"])
    return s


# ----------------------------------------------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _plain_append, "attn": _plain_attn, "commit": _plain_commit}[op](s)
    from reject_row_vocab_gb300 import specverify as sv
    if op == "attn":
        o = sv.paged_attention(s["q"], s["cache"], s["seq_lens"], max_len=s["max_len"], cu_seqlens=s["cu"],
                               row_slots=s["slots"], mask=s["mask"], scale=s["scale"], out=s["out"], ws=s["ws"])
        return {"out": o.out, "lse": o.lse}
    if op == "commit":
        sv.kv_commit(s["cache"], s["cu"], s["src"], s["dst"], max_len=s["max_len"], dev_status=s["status"])
        r = sv.kv_read(s["cache"], seq_lens=s["seq_lens"], cu_seqlens=s["cu"], max_len=s["max_len"], out=s["read"])
        return {"k": r.k, "v": r.v}
    o = sv.kv_append(s["cache"], s["knew"], s["vnew"], seq_lens=s["seq_lens"], max_len=s["max_len"], cu_seqlens=s["cu"],
                     row_slots=s["slots"], positions=s["positions"], rotation=s["rotation"], q=s["q"], out=s["out"])
    if not s["case"]["packed"]:
        return {"q": o.q, "k": s["k"], "v": s["v"]}
    r = sv.kv_read(s["cache"], layer=0, seq_lens=s["seq_lens"], max_len=s["max_len"], cu_seqlens=s["cu"],
                   row_slots=s["slots"], out=s["read"])
    return {"q": o.q, "k": r.k, "v": r.v}


def _requests_of(s):
    """Each row's request, and its number in the request."""
    B, n = s["case"]["batch"], s["max_len"]
    if s["cu"] is None:
        row = torch.arange(B * n, device=DEV)
        return row // n, row % n
    cu = s["cu"].long()
    b = torch.repeat_interleave(torch.arange(B, device=DEV), cu[1:] - cu[:-1], output_size=s["q"].shape[0])
    return b, torch.arange(s["q"].shape[0], device=DEV) - cu[b]


def _plain_rotate(x, pos, s):
    """x [rows, heads, dim] with its pairs of columns turned by pos * inv_freq."""
    c = s["case"]
    n = c["pairs"]
    angle = pos.to(torch.float64)[:, None] * s["inv_freq"].to(torch.float64)  # (far positions need the bits)
    cos, sin = torch.cos(angle).to(x.dtype)[:, None], torch.sin(angle).to(x.dtype)[:, None]
    out = x.clone()
    if c["interleaved"]:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        out[..., :n], out[..., n:2 * n] = a * cos - b * sin, b * cos + a * sin
    return out


def _plain_append(s):
    c = s["case"]
    page, D, dt = c["page"], c["head_dim"], s["qkv"].dtype
    b, j = _requests_of(s)
    at = s["seq_lens"][b] + j
    pos = at if s["positions"] is None else s["positions"]
    slot = s["slots"] if s["slots"] is not None else s["table"].long()[b, at // page] * page + at % page
    q = _plain_rotate(s["q"].float(), pos, s).to(dt)
    if not c["packed"]:
        k = _plain_rotate(s["knew"].float(), pos, s).to(dt)
        for cache, rows in ((s["k"], k), (s["v"], s["vnew"])):
            cache.view(-1, *cache.shape[3:])[slot] = rows
        return {"q": q, "k": s["k"], "v": s["v"]}
    parts = _parts(s["data"], page, D)
    # in 64 bits: a code hangs on which side of a border a value lies
    for i, rows in enumerate((_plain_rotate(s["knew"].double(), pos, s), s["vnew"].double())):
        code, scale, _ = _quantize(rows)
        parts[i][0].transpose(1, 2)[slot // page, slot % page] = code[..., 0::2] | (code[..., 1::2] << 4)
        parts[2 + i][0].transpose(1, 2)[slot // page, slot % page] = scale
    held = [p[0].transpose(1, 2)[slot // page, slot % page] for p in parts]
    return {"q": q, "k": _values(held[0], held[2]).to(dt), "v": _values(held[1], held[3]).to(dt)}


def _plain_commit(s):
    c = s["case"]
    page, n = c["page"], s["total"]
    b = torch.repeat_interleave(torch.arange(c["batch"], device=DEV), (s["cu"][1:] - s["cu"][:-1]).long(), output_size=n)
    pos, src = s["dst"][:n], s["src"][:n]
    dst = s["table"].long()[b, pos // page] * page + pos % page
    parts = _parts(s["data"], page, c["head_dim"])
    held = []
    for p in parts:
        p = p.transpose(2, 3)
        p[:, dst // page, dst % page] = p[:, src // page, src % page]
        held.append(p[:, dst // page, dst % page])
    return {"k": _values(held[0], held[2]).bfloat16(), "v": _values(held[1], held[3]).bfloat16()}


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
    slot = torch.where(there, slot, 0)
    kc, vc, ks, vs = [p[0].transpose(1, 2) for p in _parts(s["data"], page, D)]
    held = lambda codes, scales: _values(codes[slot // page, slot % page], scales[slot // page, slot % page])
    q = s["q"][row].float().reshape(B, n, G, H // G, D).permute(0, 2, 1, 3, 4).reshape(B, G, n * (H // G), D)
    x = (q @ held(kc, ks).permute(0, 2, 3, 1)) * s["scale"]
    x = x.reshape(B, G, n, H // G, P + n).masked_fill(~see[:, None, :, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == float("-inf"), 0.0, m))
    z = e.sum(-1, keepdim=True)
    o = e.reshape(B, G, n * (H // G), P + n) @ held(vc, vs).permute(0, 2, 1, 3)
    o = o.reshape(B, G, n, H // G, D) / torch.where(z == 0, 1.0, z)
    lse = (m + z.log())[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, n, H, D)
    lse = lse.permute(0, 2, 1, 3).reshape(B, n, H)
    return {"out": o[have].to(s["q"].dtype), "lse": lse[have]}


# ----------------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits, request by request and row by row
# ----------------------------------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "commit": _exact_commit}[case["op"]](s)


def _held_at(s, layer, slot):
    """K and V of one layer's slots in 64 bits, [slots, heads, dim], byte by byte from the blocks."""
    c = s["case"]
    page, D = c["page"], c["head_dim"]
    blocks = s["data"][layer]
    p, r = torch.div(slot, page, rounding_mode="floor"), torch.remainder(slot, page)
    col = torch.arange(D, device=DEV)
    sizes = torch.tensor(CODES, dtype=torch.float64, device=DEV)
    out = []
    for which in range(2):
        at = which * page * (D // 2) + r[:, None] * (D // 2) + col // 2
        byte = blocks[p].gather(2, at[:, None, :].expand(-1, c["kv_heads"], -1)).long()
        nib = torch.where(col % 2 == 0, byte % 16, byte // 16)
        at = page * D + which * page * (D // 16) + r[:, None] * (D // 16) + col // 16
        byte = blocks[p].gather(2, at[:, None, :].expand(-1, c["kv_heads"], -1)).long()
        exp, man = byte // 8, byte % 8
        scale = torch.where(exp == 0, man * 2.0 ** -17, (8 + man).double() * torch.exp2((exp - 18).double()))
        out.append(torch.where(nib >= 8, -1.0, 1.0) * sizes[nib % 8] * scale)
    return out


def _exact_values(x):
    """What the format holds of x [..., dim] in 64 bits: the nearest scale and the nearest codes, by search in their lists."""
    scales = torch.tensor([(b % 8) * 2.0 ** -17 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 18) for b in range(0xE3)],
                          dtype=torch.float64, device=DEV)
    sizes = torch.tensor(CODES, dtype=torch.float64, device=DEV)

    def nearest(a, grid):
        hi = torch.searchsorted(grid, a.contiguous()).clamp(1, grid.numel() - 1)
        lo = hi - 1
        up, down = grid[hi] - a, a - grid[lo]
        return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)

    y = x.double().unflatten(-1, (-1, GROUP))
    t = y.abs().amax(-1)
    # six times a scale against the maximum: no quotient is rounded
    s = scales[nearest(t, 6.0 * scales)][..., None]
    # likewise codes times the scale against the values (a scale of 0 holds nothing)
    best = torch.zeros_like(y)
    err = y.abs()
    for i in range(1, 8):
        e = (y.abs() - sizes[i] * s).abs()
        better = ((e < err) | ((e == err) & (i % 2 == 0))) & (s > 0)
        best, err = torch.where(better, sizes[i] * s, best), torch.where(better, e, err)
    return torch.where(y < 0, -best, best).flatten(-2)


def _exact_append(s):
    c = s["case"]
    lens, rows = _lengths(c)
    page, n = c["page"], c["pairs"]
    pos, slot, at = [], [], 0
    for b in range(c["batch"]):
        here = lens[b] + torch.arange(rows[b], device=DEV)
        pos.append(here if s["positions"] is None else s["positions"][at:at + rows[b]])
        slot.append(s["slots"][at:at + rows[b]] if s["slots"] is not None
                    else s["table"][b].long()[torch.div(here, page, rounding_mode="floor")] * page + torch.remainder(here, page))
        at += rows[b]
    pos, slot = torch.cat(pos), torch.cat(slot)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       pos.double()[:, None] * s["inv_freq"].double())[:, None]  # e^(i angle)

    def rotated(x):
        x = x.double()
        head = x[..., :2 * n]
        z = torch.view_as_complex((head.unflatten(-1, (n, 2)) if c["interleaved"]
                                   else torch.stack([head[..., :n], head[..., n:]], -1)).contiguous()) * turn
        z = torch.view_as_real(z)
        return torch.cat([z.flatten(-2) if c["interleaved"] else torch.cat([z[..., 0], z[..., 1]], -1), x[..., 2 * n:]], -1)

    q, k, v = rotated(s["q"]), rotated(s["knew"]), s["vnew"].double()
    if c["packed"]:
        return {"q": q, "k": _exact_values(k), "v": _exact_values(v)}
    out = {"q": q}
    for name, rows_ in (("k", k), ("v", v)):
        cache = s[name].double()
        cache[0, torch.div(slot, page, rounding_mode="floor"), torch.remainder(slot, page)] = rows_
        out[name] = cache
    return out


def _exact_commit(s):
    c = s["case"]
    src = s["src"][:s["total"]]
    out = [_held_at(s, layer, src) for layer in range(c["layers"])]  # what was there is what is moved
    return {"k": torch.stack([o[0] for o in out]), "v": torch.stack([o[1] for o in out])}


def _exact_attn(s):
    c = s["case"]
    lens, rows = _lengths(c)
    page, H, G, D = c["page"], c["heads"], c["kv_heads"], c["head_dim"]
    outs, lses, at = [], [], 0
    for b in range(c["batch"]):
        L, r = lens[b], rows[b]
        table = s["table"][b].long()
        pos = torch.arange(L + (0 if c["staged"] else r), device=DEV)
        slot = table[torch.div(pos, page, rounding_mode="floor")] * page + torch.remainder(pos, page)
        if c["staged"]:
            slot = torch.cat([slot, s["slots"][at:at + r]])
        k, v = _held_at(s, 0, slot)
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
