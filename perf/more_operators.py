"""The operators of an 8-bit paged cache, as workloads: norms of query and key heads with the rotation in the same pass,
appending keys and values to a cache held in 8 bits and reading them back, and attention over that cache.

Every tensor of tokens is [tokens, heads, dim]; the tokens of sequence b are the rows seq_start[b] .. seq_start[b + 1] - 1,
and kv_len[b] counts its cached tokens, the new ones included, so new token i of sequence b has position
kv_len[b] - (seq_start[b + 1] - seq_start[b]) + i.  Caches are [pages, page size, kv heads, dim] of codes (any strides),
int8 or e4m3; scales are fp32 [pages, page size / block, kv heads], one for each block of consecutive slots and head; a
cached value is its scale times its code.  page_table[b][p] is the page of positions p * page size and on.  A rotary
table row holds rot/2 cosines, then rot/2 sines.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}            # the largest code
LEAST = 2.0 ** -126                             # the smallest scale
EPS = 1e-6                                      # of the norms
LOG_LARGEST = math.log(2048 * 15360 * 32.0)     # head x query x key triples of the largest listed attention


def _case(op, **kw):
    base = {"op": op, "type": "f32", "heads": 32, "kv_heads": 8, "dim": 128, "tokens": 1, "batch": 1, "past": 0}
    if op != "norm":
        base |= {"codes": "int8", "block": 16, "page": 64, "heads_first": False, "ragged": False}
    if op in ("norm", "append"):
        base |= {"rot": kw.get("dim", 128), "interleaved": False, "norm": True, "q_out": kw.get("type", "f32")}
    if op == "read":
        base |= {"type": "bf16"}
    if op == "attention":
        base |= {"out": kw.get("type", "f32"), "cap": 0.0, "slopes": False, "window": 0, "prefix": 0, "docs": 0,
                 "causal": True}
    return base | kw


def listed():
    return [
        # the query and key heads of one decoded token: latency
        _case("norm", name="norm rope 1 token", past=777),
        # a prompt's queries and keys, half of each head turned, neighbouring pairs
        _case("norm", name="norm rope prompt half head", type="bf16", tokens=4097, past=9000, rot=64, interleaved=True),
        # one decode step of 16 sequences: q and k normed and turned, k and v quantised into blocks partly filled, which
        # are read back
        _case("append", name="append8 decode 16", heads=28, kv_heads=4, batch=16, past=2000, ragged=True),
        # three prompt chunks of a model without head norms, a scale for each token, codes kept [page, head, token]
        _case("append", name="append8 prompts e4m3", type="bf16", codes="e4m3", block=1, page=16, heads_first=True, batch=3,
              tokens=2500, past=500, ragged=True, norm=False),
        # a short sequence back to 16 bits: latency
        _case("read", name="read8 1x700", heads=28, kv_heads=4, tokens=700),
        # a long sequence moved to a 16-bit cache, e4m3 codes, a scale for each page
        _case("read", name="read8 1x65536", codes="e4m3", block=64, tokens=65536),
        # one decoded token over a short context: latency
        _case("attention", name="decode8 1x1000", heads=28, kv_heads=4, page=16, past=1000),
        # a decode step of 16 sequences of unequal length
        _case("attention", name="decode8 16x4096", heads=28, kv_heads=4, page=16, batch=16, past=4096, ragged=True),
        # one decoded token over a long context: the codes are read once at memory speed
        _case("attention", name="decode8 1x131072", type="bf16", past=131071),
        # verification of four drafted tokens and the one before them, scores capped, e4m3 codes, a scale for each token
        _case("attention", name="verify8 4x5x2000", type="f16", heads=28, kv_heads=4, codes="e4m3", block=1, page=16, batch=4,
              tokens=5, past=2000, ragged=True, cap=50.0),
        # three prompt chunks over contexts of some thousand tokens
        _case("attention", name="chunk8 3x512x4096", type="bf16", heads=28, kv_heads=4, page=16, batch=3, tokens=512, past=4096,
              ragged=True),
        # the last chunk of a long prompt, e4m3 codes
        _case("attention", name="chunk8 2048x14336", type="bf16", codes="e4m3", tokens=2048, past=14336),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "read", "attention", "attention", "attention"])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8]) if kv_heads < 16 else 16
    dim = rng.choice([64, 64, 80, 96, 112, 128, 128, 128])
    typ = rng.choice(["f32", "bf16", "f16"])
    turned = dict(rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.5, q_out=rng.choice(["f32", "bf16", typ]))
    shared = dict(type=typ, heads=heads, kv_heads=kv_heads, dim=dim)
    if op == "norm":
        return _case("norm", tokens=_log(rng, 1, 4096), past=_log(rng, 1, 16000), **turned, **shared)
    page = rng.choice([16, 16, 32, 64, 128, 48])
    shared |= dict(page=page, codes=rng.choice(["int8", "e4m3"]), heads_first=rng.random() < 0.4, ragged=rng.random() < 0.7,
                   block=rng.choice([b for b in (1, 4, 16, 16, 64) if page % b == 0]))
    batch = _log(rng, 1, 64)
    if op == "append":
        return _case("append", batch=batch, tokens=_log(rng, 1, max(1, 6000 // batch)), past=_log(rng, 1, 3000),
                     norm=rng.random() < 0.6, **turned, **shared)
    if op == "read":
        return _case("read", batch=batch, tokens=_log(rng, 1, max(1, 400000 // (batch * kv_heads))), past=rng.choice([0, 5, 300]),
                     **shared)
    tokens = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 1024)])
    past = _log(rng, 1, 60000)
    while (math.log(float(batch) * tokens * (past + tokens) * heads) > LOG_LARGEST - 0.7
           or batch * (past + tokens) * kv_heads > 1000000):
        batch, past = max(1, batch // 2), max(1, past // 2 if batch == 1 else past)
        tokens = max(1, tokens // 2) if past == 1 else tokens
    return _case("attention", out=typ, batch=batch, tokens=tokens, past=past, cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                 slopes=rng.random() < 0.2, window=rng.choice([0, 0, 0, _log(rng, 8, 4096)]),
                 prefix=rng.choice([0, 0, _log(rng, 1, 200)]), docs=rng.choice([0, 0, 0, 3]), causal=rng.random() < 0.85,
                 **shared)


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


def _tails(case):
    """Tokens of each sequence's blocks that an append touches: its new ones and those before them in their first block."""
    return [n + p % case["block"] for n, p in zip(*_lengths(case))]


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    new, past = _lengths(case)
    t, e, dim, kvh = sum(new), size[case["type"]], case["dim"], case["kv_heads"]
    if case["op"] == "norm":
        vals = t * (case["heads"] + kvh) * dim
        return {"bytes": vals * (e + size[case["q_out"]]) + t * (4 + 4 * case["rot"]), "flops": 7 * vals}
    if case["op"] == "append":
        kv, q, tail = t * kvh * dim, t * case["heads"] * dim, sum(_tails(case))
        scales = sum(-(-n // case["block"]) for n in _tails(case)) * kvh * 2 * 4
        back = 2 * tail * kvh * dim * (1 + 2) + scales
        return {"bytes": 2 * kv * (e + 1) + scales + q * (e + size[case["q_out"]]) + t * (4 + 4 * case["rot"]) + back,
                "flops": 7 * q + 10 * kv}
    if case["op"] == "read":
        vals = 2 * t * kvh * dim
        return {"bytes": vals * (1 + e) + 2 * 4 * kvh * sum(-(-n // case["block"]) for n in new), "flops": vals}
    ranges, rows, at = _visible(case), 0, 0
    for n in new:
        part = ranges[at:at + n]
        rows += max(0, max(h for _, h in part) - min(l for l, _ in part))
        at += n
    pairs = sum(h - l for l, h in ranges)
    return {"bytes": t * case["heads"] * dim * (e + size[case["out"]]) + rows * kvh * 2 * dim + rows * kvh * 8 // case["block"],
            "flops": 4 * pairs * case["heads"] * dim}


def _table(rows, rot, device):
    """cos and sin of position * 10000^(-2i/rot), formed in 64 bits, kept in 32."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _encode(x, inv, codes):
    """x times inv (32 bits) as codes."""
    y = (x * inv).clamp(-TOP[codes], TOP[codes])
    return y.round().to(torch.int8) if codes == "int8" else y.to(torch.float8_e4m3fn)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    s, typ, dim, kvh = {"case": dict(case)}, DTYPES[case["type"]], case["dim"], case["kv_heads"]
    new, past = _lengths(case)
    t = sum(new)
    # channels of unequal size, as keys have them
    spread = torch.exp(normal(kvh, dim, std=0.5))
    if case["op"] in ("norm", "append"):
        s["q_weight"] = 1.0 + normal(dim, std=0.3) if case["norm"] else None
        s["k_weight"] = 1.0 + normal(dim, std=0.3) if case["norm"] else None
        s["q"] = normal(t, case["heads"], dim, dtype=typ)
        s["k"] = (normal(t, kvh, dim) * spread).to(typ)
    if case["op"] == "norm":
        s["pos"] = (torch.arange(t, device=dev) + case["past"]).to(torch.int32)
        s["table"] = _table(t + case["past"], case["rot"], dev)
        return s
    # the cache: the sequences' pages in shuffled order among some that belong to others
    page, block, total = case["page"], case["block"], [n + p for n, p in zip(new, past)]
    counts = [-(-l // page) for l in total]
    pages = sum(counts) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(case["batch"], max(counts), dtype=torch.int32, device=dev)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    for name in ("k", "v"):
        x = normal(pages, page, kvh, dim) * (spread if name == "k" else 1.0)
        blocks = x.view(pages, page // block, block, kvh, dim)
        scale = (blocks.abs().amax((2, 4)) / TOP[case["codes"]]).clamp(min=LEAST)
        c = _encode(blocks, (1.0 / scale)[:, :, None, :, None], case["codes"]).view(pages, page, kvh, dim)
        s[name + "_cache"] = c.transpose(1, 2).contiguous().transpose(1, 2) if case["heads_first"] else c
        s[name + "_scale"] = scale
    s["page_table"] = table
    s["seq_start"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device=dev)
    s["kv_len"] = torch.tensor(total, dtype=torch.int32, device=dev)
    s["tokens"] = t
    if case["op"] == "append":
        s["v"] = normal(t, kvh, dim, dtype=typ)
        s["table"] = _table(max(total), case["rot"], dev)
        tails = _tails(case)
        s["tail_start"] = torch.tensor([sum(tails[:b]) for b in range(len(tails) + 1)], dtype=torch.int32, device=dev)
        s["tail_tokens"] = sum(tails)
    if case["op"] == "attention":
        # scores of a standard deviation of about two
        s["q"] = (normal(t, case["heads"], dim, std=2.0) / spread.repeat_interleave(case["heads"] // kvh, 0)).to(typ)
        s["slopes"] = s["prefix_len"] = s["kv_start"] = None
        if case["slopes"]:
            s["slopes"] = 2.0 ** (-8.0 * (torch.arange(case["heads"], device=dev) + 1.0) / case["heads"])
        if case["prefix"]:
            s["prefix_len"] = torch.full((case["batch"],), case["prefix"], dtype=torch.int32, device=dev)
        if case["docs"]:
            s["kv_start"] = torch.tensor(_doc_starts(case), dtype=torch.int32, device=dev)
    return s


def _normed(x, weight):
    x = x.float()
    return x if weight is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


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


def _places(start, kv_len, t):
    """Sequence and position of every token row."""
    start = start.long()
    row = torch.arange(t, device=start.device)
    seq = torch.searchsorted(start, row, right=True) - 1
    return seq, row - start[seq + 1] + kv_len.long()[seq]


def _plain_norm(s):
    c, cs = s["case"], s["table"][s["pos"].long()]
    return {n: _rotate(_normed(s[n], s[n + "_weight"]), cs, c["interleaved"]).to(DTYPES[c["q_out"]]) for n in ("q", "k")}


def _values(s, name, seq, pos):
    """Cached values of positions, in 32 bits."""
    c = s["case"]
    page, slot = s["page_table"].long()[seq, pos // c["page"]], pos % c["page"]
    return s[name + "_cache"][page, slot].float() * s[name + "_scale"][page, slot // c["block"]][..., None]


def _plain_append(s):
    c = s["case"]
    size, block, codes = c["page"], c["block"], c["codes"]
    seq, pos = _places(s["seq_start"], s["kv_len"], s["tokens"])
    cs = s["table"][pos]
    page, slot = s["page_table"].long()[seq, pos // size], pos % size
    past = s["kv_len"].long() - (s["seq_start"][1:] - s["seq_start"][:-1]).long()
    # the sequences' first blocks, and their older slots
    first_page, first = s["page_table"].long().gather(1, past[:, None] // size)[:, 0], past % size // block
    older = torch.arange(block, device=pos.device) < (past % block)[:, None]
    new = {"k": _rotate(_normed(s["k"], s["k_weight"]), cs, c["interleaved"]), "v": s["v"].float()}
    for name, x in new.items():
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        before = scale[first_page, first]
        most = torch.zeros_like(scale)
        most[first_page, first] = before * (past % block > 0)[:, None]
        where = (page * scale.shape[1] + slot // block)[:, None].expand(-1, x.shape[1])
        amax = (x.abs().amax(-1) / TOP[codes]).clamp(min=LEAST)
        most = most.view(-1, x.shape[1]).scatter_reduce(0, where, amax, "amax").view_as(scale)
        scale[page, slot // block] = most[page, slot // block]
        after = scale[first_page, first]
        ratio = before * (1.0 / after)
        rows = first_page[:, None], first[:, None] * block + torch.arange(block, device=pos.device)
        old = cache[rows].float()
        grown = older[:, :, None, None] & (after != before)[:, None, :, None]
        cache[rows] = torch.where(grown, _encode(old, ratio[:, None, :, None], codes).float(), old).to(cache.dtype)
        cache[page, slot] = _encode(x, (1.0 / scale[page, slot // block])[..., None], codes)
    q = _rotate(_normed(s["q"], s["q_weight"]), cs, c["interleaved"]).to(DTYPES[c["q_out"]])
    at = _places(s["tail_start"], s["kv_len"], s["tail_tokens"])
    return {"q": q, "k": _values(s, "k", *at).to(torch.bfloat16), "v": _values(s, "v", *at).to(torch.bfloat16)}


def _plain_read(s):
    at = _places(s["seq_start"], s["kv_len"], s["tokens"])
    return {n: _values(s, n, *at).to(DTYPES[s["case"]["type"]]) for n in ("k", "v")}


def _plain_attention(s):
    c = s["case"]
    q = s["q"].float()
    t, heads, dim = q.shape
    kvh, group, batch, most = c["kv_heads"], heads // c["kv_heads"], c["batch"], c["tokens"]
    seq, pos = _places(s["seq_start"], s["kv_len"], t)
    within = torch.arange(t, device=q.device) - s["seq_start"].long()[seq]
    # queries padded to [batch, kv head, group, new, dim]; keys and values gathered to [batch, kv head, length, dim]
    qp = q.new_zeros(batch, most, heads, dim)
    qp[seq, within] = q
    qp = qp.view(batch, most, kvh, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, kvh, group * most, dim)
    k, v = ((s[n + "_cache"].float() * s[n + "_scale"].repeat_interleave(c["block"], 1)[..., None])[s["page_table"].long()]
            .flatten(1, 2).permute(0, 2, 1, 3) for n in ("k", "v"))
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
        return {"norm": _plain_norm, "append": _plain_append, "read": _plain_read, "attention": _plain_attention}[c["op"]](s)
    import q4_dequant_gemv_gb300 as q4k
    if c["op"] == "norm":
        q, k = q4k.norm_rope(s["q"], s["k"], s["pos"], s["table"], s["q_weight"], s["k_weight"], eps=EPS,
                             interleaved=c["interleaved"], out_dtype=DTYPES[c["q_out"]])
        return {"q": q, "k": k}
    cache = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"]
    if c["op"] == "append":
        q = q4k.kv_append8(s["k"], s["v"], *cache, s["seq_start"], s["kv_len"], table=s["table"], interleaved=c["interleaved"],
                           q=s["q"], q_dtype=DTYPES[c["q_out"]], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
        k, v = q4k.kv_read8(*cache, s["tail_start"], s["kv_len"], s["tail_tokens"], dtype=torch.bfloat16)
        return {"q": q, "k": k, "v": v}
    if c["op"] == "read":
        k, v = q4k.kv_read8(*cache, s["seq_start"], s["kv_len"], s["tokens"], dtype=DTYPES[c["type"]])
        return {"k": k, "v": v}
    return q4k.paged_attention8(s["q"], *cache, s["seq_start"], s["kv_len"], out_dtype=DTYPES[c["out"]], softcap=c["cap"],
                                slopes=s["slopes"], window=c["window"], causal=c["causal"], prefix_len=s["prefix_len"],
                                kv_start=s["kv_start"])


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence."""
    s = prepare(case, seed)
    new, past = _lengths(case)

    def turned(x, pos, weight):
        """Heads over their root mean square, pairs as complex numbers times cos + i sin of the table."""
        x = x.double()
        if weight is not None:
            x = x * weight.double() * (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).rsqrt()
        row, rot = s["table"][pos].double(), case["rot"]
        turn = torch.complex(row[:, :rot // 2], row[:, rot // 2:])[:, None]
        head = x[..., :rot]
        pair = head.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., rot:]], -1)

    if case["op"] == "norm":
        return {n: turned(s[n], s["pos"].long(), s[n + "_weight"]) for n in ("q", "k")}
    page, block = case["page"], case["block"]

    def cached(name, b, upto):
        """Codes [upto, heads, dim] and scales [upto, heads] of a sequence's first positions."""
        used = s["page_table"][b, :-(-upto // page)].long()
        scale = s[name + "_scale"][used].double().repeat_interleave(block, 1).flatten(0, 1)
        return s[name + "_cache"][used].double().flatten(0, 1)[:upto], scale[:upto]

    def nearest(y):
        """The code next to y, ties to the even one."""
        if case["codes"] == "int8":
            return y.round().clamp(-127, 127)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return ((y / step).round() * step).clamp(-448, 448)

    if case["op"] == "append":
        outs, at = {"q": [], "k": [], "v": []}, 0
        for b, (n, p) in enumerate(zip(new, past)):
            pos = torch.arange(p, p + n, device=s["q"].device)
            outs["q"].append(turned(s["q"][at:at + n], pos, s["q_weight"]))
            begin = p // block * block
            for name in ("k", "v"):
                x = turned(s["k"][at:at + n], pos, s["k_weight"]) if name == "k" else s["v"][at:at + n].double()
                old, was = (y[begin:] for y in cached(name, b, p))
                every = torch.cat([torch.zeros_like(x[:p - begin]) if p - begin <= n else old * 0, x])
                width = -(-every.shape[0] // block) * block
                padded = torch.cat([every, every.new_zeros(width - every.shape[0], *every.shape[1:])])
                scale = (padded.unflatten(0, (-1, block)).abs().amax((1, 3)) / TOP[case["codes"]]).clamp(min=LEAST)
                if p > begin:
                    scale[0] = torch.maximum(scale[0], was[0])
                each = scale.repeat_interleave(block, 0)[:every.shape[0], :, None]
                vals = nearest(every / each) * each
                if p > begin:
                    kept = torch.where((scale[0] > was[0] * (1 + 1e-7))[:, None], nearest(old * (was[0] / scale[0])[:, None]), old)
                    vals[:p - begin] = kept * each[:p - begin]
                outs[name].append(vals)
            at += n
        return {name: torch.cat(v) for name, v in outs.items()}
    if case["op"] == "read":
        outs = {}
        for name in ("k", "v"):
            got = [cached(name, b, n + p) for b, (n, p) in enumerate(zip(new, past))]
            outs[name] = torch.cat([(c * e[..., None])[p:] for (c, e), p in zip(got, past)])
        return outs
    group, dim, ranges, at, ys = case["heads"] // case["kv_heads"], case["dim"], _visible(case), 0, []
    for b, (n, p) in enumerate(zip(new, past)):
        k, v = (c * e[..., None] for c, e in (cached("k", b, n + p), cached("v", b, n + p)))
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
