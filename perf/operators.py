"""The operators between a layer's q/k/v products and its output product, as workloads: rotary
positions, appending keys and values to a paged cache, and attention of new tokens over that cache.

Every tensor of tokens is [tokens, heads, dim]; the tokens of sequence b are the rows
seq_start[b] .. seq_start[b + 1] - 1, and kv_len[b] counts its cached tokens, the new ones included,
so new token i of sequence b has position kv_len[b] - (seq_start[b + 1] - seq_start[b]) + i.  Caches are
[pages, page size, kv heads, dim] (any strides); page_table[b][p] is the page of positions
p * page size and on.  A rotary table row holds rot/2 cosines, then rot/2 sines.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LOG_LARGEST = math.log(2048 * 15360 * 32.0)     # head x query x key triples of the largest listed attention


def _case(op, **kw):
    base = {"op": op, "type": "f32", "heads": 28, "kv_heads": 4, "dim": 128, "tokens": 1, "batch": 1, "past": 0}
    if op == "rope":
        base |= {"rot": 128, "interleaved": False, "long": 1.0}
    else:
        base |= {"cache": "bf16", "page": 16, "heads_first": False, "ragged": False}
    if op == "append":
        base |= {"rot": 128, "interleaved": False, "long": 1.0, "rotate_q": True, "q_out": "f32"}
    if op == "attention":
        base |= {"out": kw.get("type", "f32"), "cap": 0.0, "slopes": False, "window": 0, "prefix": 0, "docs": 0,
                 "causal": True}
    return base | kw


def listed():
    return [
        # the query heads of one decoded token, Qwen2.5-7B shaped: latency
        _case("rope", name="rope 1 token", tokens=1, past=777),
        # a prompt of a model that rotates half of each head, neighbouring pairs, positions stretched 4x
        _case("rope", name="rope prompt half head", type="bf16", heads=32, tokens=4097, past=9000, rot=64,
              interleaved=True, long=4.0),
        # one decode step of 16 sequences: q rotated, k rotated and stored, v stored
        _case("append", name="append decode 16", batch=16, tokens=1, past=2000, ragged=True),
        # a prompt chunk as the fp32 prefill product leaves it; q goes on as bf16
        _case("append", name="append chunk f32", tokens=2048, past=1000, q_out="bf16"),
        # three prompts into an fp16 cache kept [page, head, token], Llama-3-8B shaped, keys and values only
        _case("append", name="append prompts f16", type="f16", cache="f16", heads=32, kv_heads=8, batch=3, tokens=2500,
              past=0, page=64, heads_first=True, ragged=True, interleaved=True, rotate_q=False, q_out="f16"),
        # one decoded token over a short context: latency
        _case("attention", name="decode 1x1000", past=1000),
        # a decode step of 16 sequences of unequal length
        _case("attention", name="decode 16x4096", batch=16, past=4096, ragged=True),
        # one decoded token over a long context: the cache is read once at memory speed
        _case("attention", name="decode 1x131072", type="bf16", heads=32, kv_heads=8, past=131071, page=64),
        # verification of four drafted tokens and the one before them, scores capped, fp16 cache
        _case("attention", name="verify 4x5x2000", cache="f16", batch=4, tokens=5, past=2000, ragged=True, cap=50.0),
        # three prompt chunks over contexts of some thousand tokens
        _case("attention", name="chunk 3x512x4096", type="bf16", batch=3, tokens=512, past=4096, ragged=True),
        # the last chunk of a long prompt, Llama-3-8B shaped
        _case("attention", name="chunk 2048x14336", type="bf16", heads=32, kv_heads=8, tokens=2048, past=14336,
              page=64),
        # no shared heads, dim 64, distance bias, several documents in a sequence, a prefix seen by all
        _case("attention", name="masks 5x300x700", type="f16", cache="f16", heads=16, kv_heads=16, dim=64, batch=5,
              tokens=300, past=700, page=32, heads_first=True, ragged=True, slopes=True, prefix=40, docs=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "attention"])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8]) if kv_heads < 16 else 16
    dim = rng.choice([64, 64, 80, 96, 112, 128, 128, 128])
    typ = rng.choice(["f32", "bf16", "f16"])
    cache = typ if typ != "f32" else rng.choice(["bf16", "f16"])
    if op == "rope":
        return _case("rope", type=typ, heads=heads, dim=dim, tokens=_log(rng, 1, 4096), past=_log(rng, 1, 16000),
                     rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.5,
                     long=rng.choice([1.0, 4.0]))
    shared = dict(type=typ, cache=cache, heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 16, 32, 64, 128, 48]),
                  heads_first=rng.random() < 0.4, ragged=rng.random() < 0.7)
    if op == "append":
        batch = _log(rng, 1, 64)
        return _case("append", batch=batch, tokens=_log(rng, 1, max(1, 6000 // batch)), past=_log(rng, 1, 3000),
                     rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.5, rotate_q=rng.random() < 0.7,
                     q_out=rng.choice([typ, cache]), **shared)
    tokens = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 1024)])
    past = _log(rng, 1, 60000)
    batch = _log(rng, 1, 64)
    while (math.log(float(batch) * tokens * (past + tokens) * heads) > LOG_LARGEST - 0.7
           or batch * (past + tokens) * kv_heads > 1000000):
        batch, past = max(1, batch // 2), max(1, past // 2 if batch == 1 else past)
        tokens = max(1, tokens // 2) if past == 1 else tokens
    return _case("attention", out=typ, batch=batch, tokens=tokens, past=past,
                 cap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.2,
                 window=rng.choice([0, 0, 0, _log(rng, 8, 4096)]), prefix=rng.choice([0, 0, _log(rng, 1, 200)]),
                 docs=rng.choice([0, 0, 0, 3]), causal=rng.random() < 0.85, **shared)


def _lengths(case):
    """New tokens and past tokens of each sequence: equal, or between half and the whole of the case's."""
    new, past = [], []
    for b in range(case["batch"]):
        cut = (b * 2654435761 % 4096) / 8192.0 if case.get("ragged") else 0.0
        n = max(1, case["tokens"] - int(case["tokens"] * cut))
        new.append(n)
        past.append(max(0, case["past"] - int(case["past"] * cut * 0.9)))
    return new, past


def _doc_starts(case):
    """First visible position of every new token where a sequence holds several documents, else None."""
    if not case.get("docs"):
        return None
    starts = []
    for n, p in zip(*_lengths(case)):
        edges = [(n + p) * d // case["docs"] for d in range(case["docs"])]
        starts += [max(e for e in edges if e <= p + i) for i in range(n)]
    return starts


def _visible(case):
    """(lo, hi) of every new token: it sees the cached positions lo <= j < hi."""
    docs, ranges = _doc_starts(case), []
    for n, p in zip(*_lengths(case)):
        for i in range(n):
            hi = min(n + p, max(p + i + 1, case["prefix"])) if case["causal"] else n + p
            lo = max(docs[len(ranges)] if docs else 0, p + i + 1 - case["window"] if case["window"] else 0)
            ranges.append((lo, max(lo, hi)))
    return ranges


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    new, past = _lengths(case)
    t, e = sum(new), size[case["type"]]
    if case["op"] == "rope":
        vals = t * case["heads"] * case["dim"]
        return {"bytes": 2 * vals * e + t * (4 + 4 * case["rot"]), "flops": 3 * t * case["heads"] * case["rot"]}
    kv = t * case["kv_heads"] * case["dim"]
    if case["op"] == "append":
        q = t * case["heads"] * case["dim"] if case["rotate_q"] else 0
        turned = t * case["rot"] * (case["kv_heads"] + (case["heads"] if case["rotate_q"] else 0))
        return {"bytes": 2 * kv * (e + 2) + q * (e + size[case["q_out"]]) + t * (4 + 4 * case["rot"]),
                "flops": 3 * turned}
    ranges, rows, at = _visible(case), 0, 0
    for n in new:
        part = ranges[at:at + n]
        rows += max(0, max(h for _, h in part) - min(l for l, _ in part))
        at += n
    pairs = sum(h - l for l, h in ranges)
    return {"bytes": t * case["heads"] * case["dim"] * (e + size[case["out"]]) + rows * case["kv_heads"] * case["dim"] * 4,
            "flops": 4 * pairs * case["heads"] * case["dim"]}


def _table(rows, rot, long, device):
    """cos and sin of position / long * 10000^(-2i/rot), formed in 64 bits, kept in 32."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot) / long
    a = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, dtype, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    s, typ = {"case": dict(case)}, DTYPES[case["type"]]
    new, past = _lengths(case)
    t = sum(new)
    if case["op"] == "rope":
        s["x"] = normal(t, case["heads"], case["dim"], dtype=typ)
        s["pos"] = (torch.arange(t, device=dev) + case["past"]).to(torch.int32)
        s["table"] = _table(t + case["past"], case["rot"], case["long"], dev)
        return s
    # the cache: the sequences' pages in shuffled order among some that belong to others
    page, total = case["page"], [n + p for n, p in zip(new, past)]
    counts = [-(-l // page) for l in total]
    pages = sum(counts) + 3
    shape = (pages, case["kv_heads"], page, case["dim"]) if case["heads_first"] else (pages, page, case["kv_heads"], case["dim"])
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(case["batch"], max(counts), dtype=torch.int32, device=dev)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    ct = DTYPES[case["cache"]]
    for name in ("k_cache", "v_cache"):
        c = normal(*shape, dtype=ct)
        s[name] = c.transpose(1, 2) if case["heads_first"] else c
    s["page_table"] = table
    s["seq_start"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device=dev)
    s["kv_len"] = torch.tensor(total, dtype=torch.int32, device=dev)
    if case["op"] == "append":
        s["k"] = normal(t, case["kv_heads"], case["dim"], dtype=typ)
        s["v"] = normal(t, case["kv_heads"], case["dim"], dtype=typ)
        s["q"] = normal(t, case["heads"], case["dim"], dtype=typ) if case["rotate_q"] else None
        s["table"] = _table(max(total), case["rot"], case["long"], dev)
        return s
    # scores of a standard deviation of about two
    s["q"] = normal(t, case["heads"], case["dim"], dtype=typ, std=2.0)
    s["slopes"] = s["prefix_len"] = s["kv_start"] = None
    if case["slopes"]:
        s["slopes"] = 2.0 ** (-8.0 * (torch.arange(case["heads"], device=dev) + 1.0) / case["heads"])
    if case["prefix"]:
        s["prefix_len"] = torch.full((case["batch"],), case["prefix"], dtype=torch.int32, device=dev)
    if case["docs"]:
        s["kv_start"] = torch.tensor(_doc_starts(case), dtype=torch.int32, device=dev)
    return s


def _rotate(x, cs, interleaved):
    """x [tokens, heads, dim] in 32 bits, turned by the table rows cs [tokens, rot]."""
    rot = cs.shape[1]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    y = x.clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., first], x[..., second]
    y[..., first] = a * c - b * s
    y[..., second] = a * s + b * c
    return y


def _places(s):
    """Sequence and position of every new token."""
    t = (s["q"] if s["q"] is not None else s["k"]).shape[0]
    start = s["seq_start"].long()
    row = torch.arange(t, device=start.device)
    seq = torch.searchsorted(start, row, right=True) - 1
    return seq, row - start[seq + 1] + s["kv_len"].long()[seq]


def _plain_rope(s):
    c = s["case"]
    return _rotate(s["x"].float(), s["table"][s["pos"].long()], c["interleaved"]).to(s["x"].dtype)


def _plain_append(s):
    c = s["case"]
    seq, pos = _places(s)
    page, slot = s["page_table"].long()[seq, pos // c["page"]], pos % c["page"]
    cs = s["table"][pos]
    s["k_cache"][page, slot] = _rotate(s["k"].float(), cs, c["interleaved"]).to(s["k_cache"].dtype)
    s["v_cache"][page, slot] = s["v"].to(s["v_cache"].dtype)
    q = _rotate(s["q"].float(), cs, c["interleaved"]).to(DTYPES[c["q_out"]]) if s["q"] is not None else None
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    c = s["case"]
    q = s["q"].float()
    t, heads, dim = q.shape
    kvh, group, batch, most = c["kv_heads"], heads // c["kv_heads"], c["batch"], c["tokens"]
    seq, pos = _places(s)
    within = torch.arange(t, device=q.device) - s["seq_start"].long()[seq]
    # queries padded to [batch, kv head, group, new, dim]; keys and values gathered to [batch, kv head, length, dim]
    qp = q.new_zeros(batch, most, heads, dim)
    qp[seq, within] = q
    qp = qp.view(batch, most, kvh, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, kvh, group * most, dim)
    k = s["k_cache"][s["page_table"].long()].flatten(1, 2).permute(0, 2, 1, 3).float()
    v = s["v_cache"][s["page_table"].long()].flatten(1, 2).permute(0, 2, 1, 3).float()
    x = (qp @ k.transpose(2, 3)).view(batch, kvh, group, most, -1) * (1.0 / math.sqrt(dim))
    if c["cap"]:
        x = torch.tanh(x / c["cap"]) * c["cap"]
    at = torch.full((batch, most), -1, dtype=torch.int64, device=q.device)
    at[seq, within] = pos
    j = torch.arange(k.shape[2], device=q.device)
    if s["slopes"] is not None:
        x = x - s["slopes"].view(kvh, group, 1, 1) * (at[:, None, None, :, None] - j).abs()
    length = s["kv_len"].long()[:, None]
    hi = length.expand(batch, most)
    if c["causal"]:
        hi = at + 1
        if s["prefix_len"] is not None:
            hi = torch.minimum(torch.maximum(hi, s["prefix_len"].long()[:, None]), length)
    lo = (at + 1 - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(at)
    if s["kv_start"] is not None:
        first = torch.zeros_like(at)
        first[seq, within] = s["kv_start"].long()
        lo = torch.maximum(lo, first)
    seen = (j >= lo[..., None]) & (j < hi[..., None])
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - m)
    y = (p.view(batch, kvh, group * most, -1) @ v).view(batch, kvh, group, most, dim) / p.sum(-1, keepdim=True).clamp(min=1e-37)
    y = y.permute(0, 3, 1, 2, 4).reshape(batch, most, heads, dim)
    return y[seq, within].to(DTYPES[c["out"]])


def run(s):
    c = s["case"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "attention": _plain_attention}[c["op"]](s)
    import q4_dequant_gemv_gb300 as q4k
    if c["op"] == "rope":
        return q4k.rope(s["x"], s["pos"], s["table"], interleaved=c["interleaved"])
    if c["op"] == "append":
        q = q4k.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["seq_start"], s["kv_len"],
                          table=s["table"], interleaved=c["interleaved"], q=s["q"], q_dtype=DTYPES[c["q_out"]])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return q4k.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["seq_start"], s["kv_len"],
                               out_dtype=DTYPES[c["out"]], softcap=c["cap"], slopes=s["slopes"], window=c["window"],
                               causal=c["causal"], prefix_len=s["prefix_len"], kv_start=s["kv_start"])


def exact(case, seed):
    """The definitions in 64 bits, token by token of the lengths and sequence by sequence."""
    s = prepare(case, seed)
    new, past = _lengths(case)

    def turned(x, pos):
        """Pairs as complex numbers times cos + i sin of the table."""
        row, rot = s["table"][pos].double(), case["rot"]
        turn = torch.complex(row[:, :rot // 2], row[:, rot // 2:])[:, None]
        x = x.double()
        head = x[..., :rot]
        pair = head.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., rot:]], -1)

    if case["op"] == "rope":
        return turned(s["x"], s["pos"].long())
    page = case["page"]
    if case["op"] == "append":
        kc, vc, qs, at = s["k_cache"].double(), s["v_cache"].double(), [], 0
        for b, (n, p) in enumerate(zip(new, past)):
            pos = torch.arange(p, p + n, device=kc.device)
            where = s["page_table"][b].long()[pos // page], pos % page
            kc.index_put_(where, turned(s["k"][at:at + n], pos))
            vc.index_put_(where, s["v"][at:at + n].double())
            if s["q"] is not None:
                qs.append(turned(s["q"][at:at + n], pos))
            at += n
        return {"q": torch.cat(qs) if qs else None, "k_cache": kc, "v_cache": vc}
    group, dim, ranges, at, ys = case["heads"] // case["kv_heads"], case["dim"], _visible(case), 0, []
    for b, (n, p) in enumerate(zip(new, past)):
        used = s["page_table"][b, :-(-(n + p) // page)].long()
        k = s["k_cache"][used].double().flatten(0, 1)[:n + p]
        v = s["v_cache"][used].double().flatten(0, 1)[:n + p]
        q = s["q"][at:at + n].double()
        j = torch.arange(n + p, device=q.device)
        lo = torch.tensor([r[0] for r in ranges[at:at + n]], device=q.device)[:, None]
        hi = torch.tensor([r[1] for r in ranges[at:at + n]], device=q.device)[:, None]
        away = (torch.arange(p, p + n, device=q.device)[:, None] - j).abs()
        out = torch.empty(n, case["heads"], dim, dtype=torch.float64, device=q.device)
        for h in range(case["heads"]):
            x = torch.einsum("td,jd->tj", q[:, h], k[:, h // group]) / math.sqrt(dim)
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if s["slopes"] is not None:
                x = x - s["slopes"][h].double() * away
            x = torch.where((j >= lo) & (j < hi), x, torch.full_like(x, -math.inf))
            w = torch.softmax(x, -1)
            out[:, h] = torch.where(hi > lo, torch.einsum("tj,jd->td", w, v[:, h // group]), torch.zeros_like(out[:, h]))
        ys.append(out)
        at += n
    return torch.cat(ys)
