"""Measured cases of the paged KV-cache operators: append, attention, gather
and scatter, each in a plain form made of elementary torch operations and as
the calls a serving program makes of fp8_kv_cache_amd.paged."""
import math
import random

import torch

own = False

EPS = 1e-6
#: query heads, KV heads, head dimension, rotated dimensions: the head layouts
#: of Llama-3-8B, Qwen3-32B, Qwen3-30B-A3B and Phi-2.
HEADS = ((32, 8, 128, 128), (64, 8, 128, 128), (32, 4, 128, 128), (32, 32, 80, 32))


def _case(op, seqs, tokens, kv, heads, e5m2, page, *, ragged=False, head_major=False, window=0, norm=False):
    hq, hk, dim, rotary = heads
    return {"op": op, "seqs": seqs, "tokens": tokens, "kv": kv, "q_heads": hq, "kv_heads": hk, "dim": dim,
            "rotary": rotary, "e5m2": e5m2, "page": page, "ragged": ragged, "head_major": head_major,
            "window": window, "norm": norm}


def listed():
    llama, qwen, _, phi = HEADS
    return [
        # one user's next token over a short conversation: latency
        {"name": "attend 1 token, 777 keys", **_case("attention", 1, 1, 777, llama, False, 16)},
        # a decode step of a full batch, conversations of mixed length
        {"name": "attend 64 x 1, to 8192 keys", **_case("attention", 64, 1, 8192, llama, False, 16, ragged=True)},
        # a decode step over two long documents, cache held in E5M2
        {"name": "attend 2 x 1, 131072 E5M2", **_case("attention", 2, 1, 131072, qwen, True, 64, head_major=True)},
        # drafted tokens of 32 users scored in one step, one KV head a query head
        {"name": "attend 32 x 5, to 2047, D 80", **_case("attention", 32, 5, 2047, phi, False, 16, ragged=True)},
        # the last chunk of a long prompt's prefill
        {"name": "attend 2048 of 8192", **_case("attention", 1, 2048, 8192, llama, False, 16)},
        # chunks of two prompts in one step, lengths as they come, E5M2 cache
        {"name": "attend 2 x 1000 of 12345 E5M2", **_case("attention", 2, 1000, 12345, qwen, True, 32, ragged=True)},
        # a decode step's new keys and values, with the queries' and keys' norms
        {"name": "append 64 x 1, norms, E5M2", **_case("append", 64, 1, 2500, qwen, True, 16, ragged=True, norm=True)},
        # a whole prompt appended
        {"name": "append 8192", **_case("append", 1, 8192, 8192, llama, False, 16)},
        # a prompt's layer taken out of its pages to be compressed and sent
        {"name": "gather 8192", **_case("gather", 1, 8192, 8192, llama, False, 16)},
        # the long-context layer, E5M2
        {"name": "gather 131072 E5M2", **_case("gather", 1, 131072, 131072, qwen, True, 64, head_major=True)},
        # a few received prompts put into this machine's pages
        {"name": "scatter 5 x to 1013, D 80", **_case("scatter", 5, 1013, 1013, phi, False, 16, ragged=True)},
        # the long-context layer received
        {"name": "scatter 131072", **_case("scatter", 1, 131072, 131072, qwen, False, 64)},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "gather", "scatter"])
    heads = rng.choice(HEADS)
    more = dict(ragged=rng.random() < 0.7, head_major=rng.random() < 0.4, norm=op == "append" and rng.random() < 0.5)
    e5m2, page = rng.random() < 0.5, rng.choice([8, 16, 32, 64, 128])
    if op == "attention":
        more["window"] = _log(rng, 16, 4096) if rng.random() < 0.25 else 0
        kind = rng.choice(["token", "drafts", "chunk"])
        if kind == "token":
            seqs = _log(rng, 1, 128)
            kv, tokens = _log(rng, 33, min(131072, 500000 // seqs)), 1
        elif kind == "drafts":
            seqs, tokens = _log(rng, 1, 32), rng.randint(2, 9)
            kv = _log(rng, 33, 8192)
        else:
            seqs, tokens = rng.randint(1, 3), _log(rng, 65, 1100)
            kv = tokens + _log(rng, 1, 9000)
        return _case(op, seqs, tokens, kv, heads, e5m2, page, **more)
    tokens = _log(rng, 1, 8192 if op == "append" else 100000)
    seqs = _log(rng, 1, max(1, min(64, (8192 if op == "append" else 100000) // tokens)))
    return _case(op, seqs, tokens, tokens + (rng.randint(0, 2000) if op == "append" else 0), heads, e5m2, page, **more)


def _lengths(c):
    """New tokens and cache length of each sequence; the first has the most of both."""
    r = random.Random(c["seqs"] * 1000003 + c["tokens"] * 101 + c["kv"])
    new, kv = [], []
    for s in range(c["seqs"]):
        n = c["tokens"] if s == 0 or not c["ragged"] else r.randint(-(-c["tokens"] // 2), c["tokens"])
        lone = c["kv"] if s == 0 or not c["ragged"] else r.randint(max(n, c["kv"] // 8), max(n, c["kv"]))
        new.append(n)
        kv.append(n if c["op"] in ("gather", "scatter") else lone)
    return new, kv


def _values(g, tokens, heads, dim, outliers):
    """Heavy-tailed cache values: N(0,1) times a lognormal scale for each
    channel, four larger channels a head for keys."""
    scale = torch.exp(0.5 * torch.randn(heads, dim, generator=g, device="cuda"))
    if outliers:
        at = torch.rand(heads, dim, generator=g, device="cuda").argsort(1)[:, :4]
        scale.scatter_(1, at, 4 * scale.gather(1, at))
    return torch.randn(tokens, heads, dim, generator=g, device="cuda") * scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    new, kv = _lengths(c)
    total = sum(new)
    need = [-(-n // c["page"]) for n in kv]
    pages = sum(need) + max(2, sum(need) // 4)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)   # pages as they come after long use
    table = torch.full((c["seqs"], max(need)), -1, dtype=torch.int32, device="cuda")
    begin = torch.tensor([sum(need[:s]) for s in range(c["seqs"])], device="cuda")
    column = torch.arange(max(need), device="cuda")
    used = column < torch.tensor(need, device="cuda")[:, None]
    table[used] = order[(begin[:, None] + column)[used]]
    hk, dim, hq = c["kv_heads"], c["dim"], c["q_heads"]

    def pool(outliers):
        x = _values(g, pages * c["page"], hk, dim, outliers).to(torch.bfloat16)
        x = x.to(torch.float8_e5m2) if c["e5m2"] else x
        x = x.view(pages, c["page"], hk, dim)
        if c["head_major"]:   # a page holds each head's tokens together
            raw = x.view(torch.uint8) if c["e5m2"] else x
            raw = raw.transpose(1, 2).contiguous().transpose(1, 2)
            x = raw.view(torch.float8_e5m2) if c["e5m2"] else raw
        return x

    st = {"case": c, "k_pool": pool(True), "v_pool": pool(False), "table": table,
          "cu": torch.tensor([sum(new[:s]) for s in range(c["seqs"] + 1)], dtype=torch.int32, device="cuda"),
          "kv_lens": torch.tensor(kv, dtype=torch.int32, device="cuda"), "max_new": max(new), "max_kv": max(kv),
          "total": total}
    if c["op"] in ("append", "attention"):
        st["q"] = torch.randn(total, hq, dim, generator=g, device="cuda").to(torch.bfloat16)
    if c["op"] in ("append", "scatter"):
        st["k"] = _values(g, total, hk, dim, True).to(torch.bfloat16)
        st["v"] = _values(g, total, hk, dim, False).to(torch.bfloat16)
        if c["op"] == "scatter" and c["e5m2"]:
            st["k"], st["v"] = st["k"].to(torch.float8_e5m2), st["v"].to(torch.float8_e5m2)
    if c["op"] == "append":
        half = c["rotary"] // 2
        angle = torch.arange(max(kv), device="cuda", dtype=torch.float64)[:, None] * torch.exp(
            torch.arange(half, device="cuda", dtype=torch.float64) * (-math.log(1e6) / half))
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
        w = 1 + 0.2 * torch.randn(2, dim, generator=g, device="cuda")
        st["q_norm"], st["k_norm"] = (w[0].to(torch.bfloat16), w[1].to(torch.bfloat16)) if c["norm"] else (None, None)
    if own:   # the handles that a program keeps for its cache and for a step's batch
        from fp8_kv_cache_amd import paged
        st["cache"] = paged.PagedCache(st["k_pool"], st["v_pool"])
        st["batch"] = paged.PageBatch(table, st["cu"], st["kv_lens"], total, st["max_new"], st["max_kv"])
        st["rope"] = paged.Rope(st["cos_sin"]) if c["op"] == "append" else None
    return st


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        from fp8_kv_cache_amd import paged
        if op == "attention":
            out, lse = paged.attention(st["cache"], st["batch"], st["q"], window=st["case"]["window"], return_lse=True)
            return {"out": out, "lse": lse}
        if op == "append":
            q = paged.append(st["cache"], st["batch"], st["k"], st["v"], q=st["q"], rope=st["rope"],
                             q_norm=st["q_norm"], k_norm=st["k_norm"], eps=EPS)
            return {"q": q, "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
        if op == "gather":
            k, v = paged.gather(st["cache"], st["batch"])
            return {"k": k, "v": v}
        paged.scatter(st["cache"], st["batch"], st["k"], st["v"])
        return {"k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    if op == "attention":
        return _plain_attention(st)
    seq, position = _tokens(st)
    page = st["table"][seq, position // st["case"]["page"]].long()
    slot = position % st["case"]["page"]
    if op == "gather":
        return {"k": _bits(st["k_pool"])[page, slot].view(st["k_pool"].dtype),
                "v": _bits(st["v_pool"])[page, slot].view(st["v_pool"].dtype)}
    k, v = st["k"], st["v"]
    if op == "append":
        k = _plain_rotate(_plain_norm(k.float(), st["k_norm"]), st["cos_sin"][position])
        q = _plain_rotate(_plain_norm(st["q"].float(), st["q_norm"]), st["cos_sin"][position])
        k, v = k.to(st["k_pool"].dtype), v.to(st["v_pool"].dtype)
    _bits(st["k_pool"])[page, slot] = _bits(k)
    _bits(st["v_pool"])[page, slot] = _bits(v)
    out = {"k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    return {"q": q.to(torch.bfloat16), **out} if op == "append" else out


def _bits(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e5m2 else x


def _tokens(st):
    """Sequence and position of each new token."""
    row = torch.arange(st["total"], device="cuda")
    seq = torch.bucketize(row, st["cu"][1:].long(), right=True)
    new = (st["cu"][1:] - st["cu"][:-1]).long()
    return seq, st["kv_lens"].long()[seq] - new[seq] + row - st["cu"].long()[seq]


def _plain_norm(x, w):
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _plain_rotate(x, cos_sin):
    half = cos_sin.shape[1] // 2
    cos, sin = cos_sin[:, None, :half], cos_sin[:, None, half:]
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _plain_attention(st):
    c = st["case"]
    seqs, hk, dim = c["seqs"], c["kv_heads"], c["dim"]
    group, most, length = c["q_heads"] // hk, st["max_new"], st["max_kv"]
    key = torch.arange(length, device="cuda")
    kv = st["kv_lens"].long()[:, None]
    there = key < kv
    page = torch.where(there, st["table"][:, key // c["page"]].long(), 0)
    slot = (key % c["page"]).expand(seqs, length)
    k = _bits(st["k_pool"])[page, slot].view(st["k_pool"].dtype).float()           # sequence, key, head, dim
    v = _bits(st["v_pool"])[page, slot].view(st["v_pool"].dtype).float()
    i = torch.arange(most, device="cuda")
    new = (st["cu"][1:] - st["cu"][:-1]).long()[:, None]
    row = (st["cu"][:-1].long()[:, None] + i).clamp(max=st["total"] - 1)
    q = st["q"][row].float().view(seqs, most, hk, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs * hk, group * most, dim)
    k = k.permute(0, 2, 3, 1).reshape(seqs * hk, dim, length).contiguous()
    v = v.masked_fill(~there[:, :, None, None], 0).permute(0, 2, 1, 3).reshape(seqs * hk, length, dim).contiguous()
    position = kv - new + i                                                         # sequence, token
    seen = key <= position[:, :, None]
    if c["window"]:
        seen &= key > position[:, :, None] - c["window"]
    score = torch.bmm(q, k).view(seqs, hk, group, most, length) * (1 / math.sqrt(dim))
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp_(score.sub_(torch.where(top == -math.inf, 0, top)))
    total = weight.sum(-1, keepdim=True)
    out = torch.bmm(weight.view(seqs * hk, group * most, length), v).view(seqs, hk, group, most, dim)
    out = torch.where(total > 0, out / total, 0)
    lse = (torch.log(total) + top)[..., 0]
    seq = torch.bucketize(torch.arange(st["total"], device="cuda"), st["cu"][1:].long(), right=True)
    at = torch.arange(st["total"], device="cuda") - st["cu"].long()[seq]
    out = out.permute(0, 3, 1, 2, 4).reshape(seqs, most, c["q_heads"], dim)[seq, at]
    return {"out": out.to(torch.bfloat16), "lse": lse.permute(0, 3, 1, 2).reshape(seqs, most, c["q_heads"])[seq, at]}


def _seen_pairs(c):
    """Query-key pairs inside the mask, and keys that any query sees, over all sequences."""
    pairs = keys = 0
    for n, kv in zip(*_lengths(c)):
        first = kv - n
        if c["window"]:
            w = c["window"]
            full = max(0, kv - max(first, w))              # positions that see w keys
            short = max(0, min(kv, w) - first)             # positions p < w that see p + 1
            pairs += full * w + sum(range(first + 1, first + 1 + short))
            keys += kv - max(0, first + 1 - w)
        else:
            pairs += n * first + n * (n + 1) // 2
            keys += kv
    return pairs, keys


def work(case):
    c = case
    new, kv = _lengths(c)
    total, size = sum(new), 1 if c["e5m2"] else 2
    row = c["kv_heads"] * c["dim"]
    tables = 4 * (sum(-(-x // c["page"]) for x in kv) + 2 * c["seqs"] + 1)
    if c["op"] == "attention":
        pairs, keys = _seen_pairs(c)
        q = total * c["q_heads"] * c["dim"]
        return {"bytes": 2 * keys * row * size + 4 * q + 4 * total * c["q_heads"] + tables,
                "flops": 4 * pairs * c["q_heads"] * c["dim"]}
    if c["op"] == "append":
        q = total * c["q_heads"] * c["dim"]
        return {"bytes": 4 * q + 2 * total * row * (2 + size) + 4 * total * c["rotary"] + tables,
                "flops": total * (c["q_heads"] + c["kv_heads"]) * (3 * c["rotary"] + (4 * c["dim"] if c["norm"] else 0))}
    return {"bytes": 4 * total * row * size + tables, "flops": 0}


def exact(case, seed):
    """From the definitions, sequence by sequence, in 64 bits."""
    c, st = case, prepare(case, seed)
    new, kv = _lengths(c)
    table = st["table"].long()
    rows = c["page"]

    def where(s, positions):
        return table[s][positions // rows], positions % rows

    def values(x):
        return x.to(torch.float64)

    begin = 0
    if c["op"] == "gather":
        parts = []
        for s, n in enumerate(new):
            page, slot = where(s, torch.arange(kv[s] - n, kv[s], device="cuda"))
            parts.append((values(st["k_pool"])[page, slot], values(st["v_pool"])[page, slot]))
        return {"k": torch.cat([p[0] for p in parts]), "v": torch.cat([p[1] for p in parts])}
    if c["op"] in ("append", "scatter"):
        k_pool, v_pool = values(st["k_pool"]), values(st["v_pool"])
        q_rows = []
        for s, n in enumerate(new):
            at = torch.arange(kv[s] - n, kv[s], device="cuda")
            page, slot = where(s, at)
            k, v = values(st["k"][begin:begin + n]), values(st["v"][begin:begin + n])
            if c["op"] == "append":
                k = _exact_position(k, st["k_norm"], st["cos_sin"], at)
                q_rows.append(_exact_position(values(st["q"][begin:begin + n]), st["q_norm"], st["cos_sin"], at))
            k_pool[page, slot] = k
            v_pool[page, slot] = v
            begin += n
        out = {"k_pool": k_pool, "v_pool": v_pool}
        return {"q": torch.cat(q_rows), **out} if c["op"] == "append" else out
    group = c["q_heads"] // c["kv_heads"]
    out = torch.zeros(st["total"], c["q_heads"], c["dim"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["total"], c["q_heads"], dtype=torch.float64, device="cuda")
    for s, n in enumerate(new):
        first = kv[s] - n
        low = max(0, first + 1 - c["window"]) if c["window"] else 0
        at = torch.arange(low, kv[s], device="cuda")
        page, slot = where(s, at)
        query_at = torch.arange(first, kv[s], device="cuda")[:, None]
        hidden = at > query_at
        if c["window"]:
            hidden |= at <= query_at - c["window"]
        keys, vals = values(_bits(st["k_pool"])[page, slot].view(st["k_pool"].dtype)), values(
            _bits(st["v_pool"])[page, slot].view(st["v_pool"].dtype))
        for h in range(c["q_heads"]):
            q = values(st["q"][begin:begin + n, h])
            score = (q @ keys[:, h // group].T.contiguous()) / math.sqrt(c["dim"])
            score[hidden] = -math.inf
            lse[begin:begin + n, h] = torch.logsumexp(score, 1)
            out[begin:begin + n, h] = torch.softmax(score, 1) @ vals[:, h // group].contiguous()
        begin += n
    return {"out": out, "lse": lse}


def _exact_position(x, w, cos_sin, at):
    """Norm and rotation of x [tokens, heads, dim] by complex products."""
    if w is not None:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.to(torch.float64)
    half = cos_sin.shape[1] // 2
    turn = torch.complex(cos_sin[at, :half].to(torch.float64), cos_sin[at, half:].to(torch.float64))[:, None]
    z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn
    return torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)
