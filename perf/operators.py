"""Cases of the decode-side operators on rotated queries and keys and the paged cache.

Three operators: the norm of every query and key head with the position rotation in one pass
(`rotate`), keys and values appended to a paged cache with that pass on the way (`append`), and
attention for a batch that shares a long prefix in that cache, computed once for the batch, with
each sequence's own pages behind it (`attend`).  Everything is seeded; the cache's pages are handed
out in random order, as a serving program's allocator does.
"""
import math

import torch

own = False

#: steps of the golden ratio spread the lengths of a case, the same for every seed
GOLDEN = 0.6180339887498949
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------
# Cases
def listed():
    rot = dict(op="rotate", kv_heads=8, group=4, d=128, dtype="bf16", rotary=128, interleaved=False,
               norm=True, base=1e6, far=131072)
    app = dict(op="append", kv_heads=8, group=4, d=128, dtype="bf16", rotary=128, interleaved=False,
               norm=True, base=1e6, page=64, far=131072)
    att = dict(op="attend", kv_heads=8, group=4, d=128, dtype="bf16", page=64, groups=1, q_max=1,
               prefix=0, tail=0, tail_min=1, prior=False)
    return [
        # one decode token of each of eight sequences: a launch's latency
        dict(rot, name="rotate decode b8", tokens=8),
        # heads rotated on half their channels in pairs, an odd number of tokens of a packed batch
        dict(rot, name="rotate ragged", tokens=1021, kv_heads=2, group=8, d=64, dtype="fp16", rotary=32,
             interleaved=True, norm=False, base=1e4, far=8192),
        # a 32K prompt, from the fused projection's rows
        dict(rot, name="rotate prompt 32k", tokens=32768),
        # a decode step: queries and keys normalised and rotated, the token appended to its page
        dict(app, name="append decode b8", seqs=8, new=1, page=16, with_q=True),
        # drafted tokens, a few for each of many sequences
        dict(app, name="append drafts", seqs=111, new=7, kv_heads=2, group=8, d=64, dtype="fp16", page=32,
             norm=False, rotary=64, base=1e4, far=8192, with_q=True),
        # four prompts of 8192 tokens entering the cache (their queries go another way)
        dict(app, name="append prompts 4x8k", seqs=4, new=8192, with_q=False),
        # the tokens decoded so far behind a compressed context whose attention is at hand
        dict(att, name="attend tails b8", seqs=8, tail=512, page=16, prior=True),
        # drafted tokens, two prefixes, ragged tails
        dict(att, name="attend drafts", seqs=34, groups=2, q_max=5, kv_heads=2, group=8, d=64, dtype="fp16",
             page=32, prefix=8191, tail=2039, tail_min=7),
        # a decode step of eight sequences behind one 32K prompt
        dict(att, name="attend prefix 32k b8", seqs=8, prefix=32768, tail=512),
        # four sequences behind 128K
        dict(att, name="attend prefix 128k b4", seqs=4, prefix=131072, tail=1024),
        # nothing shared: paged decode over ragged contexts
        dict(att, name="attend paged b32", seqs=32, tail=16384, tail_min=100),
        # a wide batch behind one 32K prompt: the prefix is a matrix product
        dict(att, name="attend prefix 32k b256", seqs=256, prefix=32768, tail=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128])
    c = dict(op=rng.choice(["rotate", "append", "attend", "attend"]), kv_heads=rng.choice([1, 2, 4, 8]),
             group=rng.choice([1, 2, 4, 8]), d=d, dtype=rng.choice(["bf16", "fp16"]))
    if c["op"] == "attend":
        while True:
            g = rng.choice([1, 1, 1, 2, 3])
            a = dict(c, page=rng.choice([16, 32, 64, 128, 256]), groups=g, seqs=g * _log(rng, 1, 256 // g),
                     q_max=rng.choice([1, 1, 1, 2, 5, 8]), prefix=rng.choice([0, 1, 1]) * _log(rng, 33, 131072),
                     tail=_log(rng, 1, 16384), tail_min=0, prior=rng.choice([False, True]))
            scores = a["seqs"] * a["q_max"] * a["kv_heads"] * a["group"] * (a["prefix"] + a["tail"])
            cached = (g * a["prefix"] + a["seqs"] * a["tail"]) * a["kv_heads"] * d
            if scores <= 256 * 32 * 32768 and cached <= 32 * 16384 * 8 * 128 and a["prefix"] + a["tail"] > 8:
                a["tail_min"] = min(a["tail"], rng.choice([0, 1, 9]))
                return a
    c |= dict(rotary=rng.choice([d, d, d // 2]), interleaved=rng.choice([False, True]), norm=rng.choice([True, False]),
              base=rng.choice([1e4, 1e6]), far=rng.choice([8192, 131072]))
    if c["op"] == "rotate":
        return dict(c, tokens=_log(rng, 1, 32768))
    seqs = _log(rng, 1, 256)
    return dict(c, page=rng.choice([16, 32, 64, 128, 256]), seqs=seqs, new=_log(rng, 1, 32768 // seqs),
                with_q=rng.choice([True, False]))


def _spread(count, lo, hi):
    """`count` whole numbers spread over lo .. hi, in no order, with lo and hi among them if there is room."""
    got = [lo + int((hi - lo + 1) * ((i * GOLDEN) % 1.0)) for i in range(count)]
    got[-1] = hi
    return got


def _attend_sizes(c):
    """Queries of each sequence (1 .. q_max), cached tokens behind its prefix, prefix of each group."""
    qs = _spread(c["seqs"], 1, c["q_max"])
    tails = _spread(c["seqs"], c["tail_min"], c["tail"]) if c["tail"] else [0] * c["seqs"]
    prefixes = [max(0, c["prefix"] - 37 * g) for g in range(c["groups"])] if c["prefix"] else [0] * c["groups"]
    return qs, tails, prefixes


# ------------------------------------------------------------------------------------------------
# Inputs
def _randn(shape, dtype, gen):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=gen)


def _inv_freq(c):
    i = torch.arange(0, c["rotary"], 2, dtype=torch.float64, device="cuda")
    return c["base"] ** (-i / c["rotary"])


def _channel_scales(d, dtype):
    """Keys have a few channels far larger than the rest."""
    s = torch.ones(d, dtype=dtype, device="cuda")
    s[:: d // 4] = 8.0
    s[3 :: d // 4] = 4.0
    return s


def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    h, g, d = c["kv_heads"], c["group"], c["d"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": c, "dtype": dt}
    if c["op"] in ("rotate", "append"):
        tokens = c["tokens"] if c["op"] == "rotate" else c["seqs"] * c["new"]
        # the projection's rows: queries, keys and values of a token behind one another
        qkv = _randn((tokens, h * g + 2 * h, d), dt, gen)
        qkv[:, h * g : h * g + h] *= _channel_scales(d, dt)
        s["q"], s["k"], s["v"] = qkv[:, : h * g], qkv[:, h * g : h * g + h], qkv[:, h * g + h :]
        s["wq"] = (1 + 0.2 * _randn((d,), torch.float32, gen)).to(dt) if c["norm"] else None
        s["wk"] = (1 + 0.2 * _randn((d,), torch.float32, gen)).to(dt) if c["norm"] else None
        s["inv_freq"] = _inv_freq(c)
    if c["op"] == "rotate":
        # a packed batch: positions run on to a far one, whatever token comes first
        s["positions"] = ((torch.arange(tokens, device="cuda") * 7919 + seed * 104729) % c["far"]).to(torch.int32)
    if c["op"] == "append":
        per = c["new"] // c["page"] + 2  # pages of a sequence: its new tokens start inside a page
        s["kv"] = torch.zeros((1, c["seqs"] * per, h, c["page"], 2, d), dtype=dt, device="cuda")
        s["table"] = torch.randperm(c["seqs"] * per, device="cuda", generator=gen).to(torch.int32).view(c["seqs"], per)
        first = torch.randint(0, c["page"], (c["seqs"],), device="cuda", generator=gen)
        s["seq"] = torch.arange(c["seqs"], device="cuda", dtype=torch.int32).repeat_interleave(c["new"])
        s["index"] = (first[:, None] + torch.arange(c["new"], device="cuda")).reshape(-1).to(torch.int32)
        behind = torch.randint(0, c["far"], (c["seqs"],), device="cuda", generator=gen)  # tokens before its pages
        s["positions"] = (s["index"] + behind.repeat_interleave(c["new"])).to(torch.int32)
    if c["op"] == "attend":
        qs, tails, prefixes = _attend_sizes(c)
        page = c["page"]
        pre_pages, own_pages = -(-max(prefixes) // page), max(1, -(-max(tails) // page))
        pages = c["groups"] * pre_pages + c["seqs"] * own_pages
        kv = _randn((1, pages, h, page, 2, d), dt, gen)
        kv[..., 0, :] *= _channel_scales(d, dt)
        order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
        s["kv"] = kv
        s["prefix_table"] = order[: c["groups"] * pre_pages].view(c["groups"], pre_pages)
        s["table"] = order[c["groups"] * pre_pages :].view(c["seqs"], own_pages)
        s["q"] = _randn((sum(qs), h * g, d), dt, gen)
        s["lengths"] = torch.tensor(tails, dtype=torch.int32, device="cuda")
        s["prefix_lengths"] = torch.tensor(prefixes, dtype=torch.int32, device="cuda")
        starts = [0]
        for n in qs:
            starts.append(starts[-1] + n)
        s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["group_start"] = torch.arange(c["groups"] + 1, dtype=torch.int32, device="cuda") * (c["seqs"] // c["groups"])
        s["max_length"], s["max_prefix"] = max(tails), max(prefixes)
        # where a query stands: its sequence and its place among that sequence's queries
        of = torch.arange(c["seqs"], device="cuda").repeat_interleave(torch.tensor(qs, device="cuda"))
        s["q_seq"], s["q_place"] = of, torch.arange(sum(qs), device="cuda") - s["q_start"][of]
        s["prior"] = None
        if c["prior"]:  # attention over tokens held elsewhere, about as much weight as the cached ones
            s["prior"] = (_randn((sum(qs), h * g, d), torch.float32, gen) * 0.05,
                          math.log(max(tails) + 1) + 1.5 + _randn((sum(qs), h * g), torch.float32, gen))
    if own:
        from verified_kv_cache_poissoncomp_gb300 import paged

        s["cache"] = paged.PagedKV(h, g, d, dtype=dt, kv=s.get("kv"))
        if "inv_freq" in s:
            s["rope"] = paged.Rope(s["inv_freq"], interleaved=c["interleaved"])
    return s


# ------------------------------------------------------------------------------------------------
# One pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    c, op = s["case"], s["case"]["op"]
    if op == "rotate":
        return s["cache"].norm_rotate(s["q"], s["k"], s["positions"], s["rope"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS)
    if op == "append":
        q = s["cache"].append(0, s["k"], s["v"], s["seq"], s["index"], s["table"], positions=s["positions"], rope=s["rope"],
                              k_weight=s["wk"], eps=EPS, q=s["q"] if c["with_q"] else None, q_weight=s["wq"])
        return s["kv"], q
    shared = {}
    if c["prefix"]:
        shared = dict(prefix_table=s["prefix_table"], prefix_lengths=s["prefix_lengths"], max_prefix=s["max_prefix"])
        if c["groups"] > 1:
            shared["group_start"] = s["group_start"]
    return s["cache"].attend(0, s["q"], s["table"], s["lengths"], s["max_length"],
                             q_start=s["q_start"] if c["q_max"] > 1 else None, prior=s["prior"], **shared)


def _normed(x, weight):
    x = x.float()
    return x if weight is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _rotated(x, s):
    """x float [tokens][heads][d], its first `rotary` channels turned by position * inv_freq."""
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r, rest = x[..., : c["rotary"]], x[..., c["rotary"] :]
    if c["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r.chunk(2, -1)
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1).to(s["dtype"])


def _run_plain(s):
    c = s["case"]
    if c["op"] == "rotate":
        return _rotated(_normed(s["q"], s["wq"]), s), _rotated(_normed(s["k"], s["wk"]), s)
    if c["op"] == "append":
        seq, index = s["seq"].long(), s["index"].long()
        page, slot = s["table"][seq, index // c["page"]].long(), index % c["page"]
        s["kv"][0, page, :, slot, 0] = _rotated(_normed(s["k"], s["wk"]), s)
        s["kv"][0, page, :, slot, 1] = s["v"]
        return s["kv"], _rotated(_normed(s["q"], s["wq"]), s) if c["with_q"] else None
    return _attend_plain(s)


def _gathered(kv, table):
    """Rows of each table's pages in order: float [tables][kv_heads][tokens][2][d]."""
    p = kv[0][table.long()]  # [tables][pages][kv_heads][page][2][d]
    return p.permute(0, 2, 1, 3, 4, 5).flatten(2, 3).float()


def _attend_plain(s):
    c = s["case"]
    h, g, d, seqs, groups, q_max = c["kv_heads"], c["group"], c["d"], c["seqs"], c["groups"], c["q_max"]
    scale = d**-0.5
    # queries padded to q_max a sequence: [seqs][kv_heads][q_max * group][d]
    padded = torch.zeros((seqs, q_max, h * g, d), dtype=torch.float32, device="cuda")
    padded[s["q_seq"], s["q_place"]] = s["q"].float()
    q = padded.view(seqs, q_max, h, g, d).transpose(1, 2).reshape(seqs, h, q_max * g, d) * scale
    own_kv = _gathered(s["kv"], s["table"])
    score = q @ own_kv[:, :, :, 0].transpose(-1, -2)
    count = s["q_start"][1:] - s["q_start"][:-1]
    last = (s["lengths"] - count)[:, None] + torch.arange(q_max, device="cuda").repeat_interleave(g)  # a query's own token
    seen = torch.arange(score.shape[-1], device="cuda") <= last[:, None, :, None]
    parts = [score.masked_fill(~(seen & (torch.arange(score.shape[-1], device="cuda") < s["lengths"][:, None, None, None])), -math.inf)]
    if c["prefix"]:
        pre = _gathered(s["kv"], s["prefix_table"])
        together = q.view(groups, seqs // groups, h, q_max * g, d).transpose(1, 2).flatten(2, 3)
        score = together @ pre[:, :, :, 0].transpose(-1, -2)
        score = score.masked_fill(torch.arange(score.shape[-1], device="cuda") >= s["prefix_lengths"][:, None, None, None], -math.inf)
        parts.append(score.view(groups, h, seqs // groups, q_max * g, -1).transpose(1, 2).reshape(seqs, h, q_max * g, -1))
    if s["prior"] is not None:
        po = torch.zeros((seqs, q_max, h * g, d), device="cuda")
        pl = torch.zeros((seqs, q_max, h * g), device="cuda")
        po[s["q_seq"], s["q_place"]], pl[s["q_seq"], s["q_place"]] = s["prior"]
        po = po.view(seqs, q_max, h, g, d).transpose(1, 2).reshape(seqs, h, q_max * g, d)
        parts.append(pl.view(seqs, q_max, h, g).transpose(1, 2).reshape(seqs, h, q_max * g, 1))
    score = torch.cat(parts, -1)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = weight.sum(-1, keepdim=True)
    at = own_kv.shape[2]
    out = weight[..., :at] @ own_kv[:, :, :, 1]
    if c["prefix"]:
        n = pre.shape[2]
        w = weight[..., at : at + n].view(groups, seqs // groups, h, q_max * g, n).transpose(1, 2).flatten(2, 3)
        out = out + (w @ pre[:, :, :, 1]).view(groups, h, seqs // groups, q_max * g, d).transpose(1, 2).reshape(out.shape)
    if s["prior"] is not None:
        out = out + weight[..., -1:] * po
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = top + torch.log(total)  # -inf where nothing is seen
    back = lambda x: x.view(seqs, h, q_max, g, -1).transpose(1, 2).flatten(2, 3)[s["q_seq"], s["q_place"]]  # noqa: E731
    return back(out).to(s["dtype"]), back(lse)[..., 0]


# ------------------------------------------------------------------------------------------------
# What a pass cannot do without
def work(case):
    c = case
    h, hq, d = c["kv_heads"], c["kv_heads"] * c["group"], c["d"]
    if c["op"] == "rotate":
        rows = c["tokens"] * (hq + h)
        return {"bytes": 2 * rows * d * 2 + 4 * c["tokens"], "flops": rows * d * (7 if c["norm"] else 3)}
    if c["op"] == "append":
        tokens = c["seqs"] * c["new"]
        rows = tokens * ((hq if c["with_q"] else 0) + 2 * h)
        return {"bytes": 2 * rows * d * 2 + 12 * tokens, "flops": (rows - tokens * h) * d * (7 if c["norm"] else 3)}
    qs, tails, prefixes = _attend_sizes(c)
    per = c["seqs"] // c["groups"]
    seen = sum(n * prefixes[i // per] + sum(max(0, tails[i] - n + 1 + j) for j in range(n)) for i, n in enumerate(qs))
    rows = sum(qs) * hq
    more = rows * (d + 1) * 4 if c["prior"] else 0
    return {"bytes": (sum(tails) + sum(prefixes)) * h * 2 * d * 2 + rows * (4 * d + 4) + more, "flops": 4 * d * hq * seen}


# ------------------------------------------------------------------------------------------------
# The definition in 64 bits
def _exact_heads(x, weight, s):
    c, t = s["case"], x.shape[0]
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["d"] + EPS) * weight.double()
    half = c["rotary"] // 2
    z = torch.polar(torch.ones((t, half), dtype=torch.float64, device="cuda"), torch.outer(s["positions"].double(), s["inv_freq"]))
    out = y.clone()
    first, second = (slice(0, c["rotary"], 2), slice(1, c["rotary"], 2)) if c["interleaved"] else (slice(0, half), slice(half, c["rotary"]))
    turned = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * z[:, None]
    out[..., first], out[..., second] = turned.real, turned.imag
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = case
    if c["op"] == "rotate":
        return _exact_heads(s["q"], s["wq"], s), _exact_heads(s["k"], s["wk"], s)
    if c["op"] == "append":
        kv = s["kv"].double()
        flat = (s["table"].long().gather(1, (s["index"].view(c["seqs"], -1) // c["page"]).long()).view(-1) * c["page"]
                + s["index"] % c["page"])
        rows = kv[0].transpose(1, 2).reshape(-1, c["kv_heads"], 2, c["d"])
        rows[flat] = torch.stack((_exact_heads(s["k"], s["wk"], s), s["v"].double()), 2)
        kv = rows.view(1, -1, c["page"], c["kv_heads"], 2, c["d"]).transpose(2, 3).contiguous()
        return kv, _exact_heads(s["q"], s["wq"], s) if c["with_q"] else None
    qs, tails, prefixes = _attend_sizes(c)
    h, g, d = c["kv_heads"], c["group"], c["d"]
    out = torch.zeros((sum(qs), h * g, d), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(qs), h * g), -math.inf, dtype=torch.float64, device="cuda")

    def rows_of(table, n):
        used = table[: -(-n // c["page"])].long()
        return s["kv"][0][used].transpose(0, 1).flatten(1, 2)[:, :n].double()  # [kv_heads][n][2][d]

    at, before = 0, None
    for i, n in enumerate(qs):
        group = i // (c["seqs"] // c["groups"])
        if before is None or before[0] != group:
            before = (group, rows_of(s["prefix_table"][group], prefixes[group]) if c["prefix"] else None)
        q = s["q"][at : at + n].double().view(n, h, g, d)
        kv = [x for x in (before[1], rows_of(s["table"][i], tails[i])) if x is not None]
        logits = [torch.einsum("nhgd,hmd->hngm", q, x[:, :, 0]) / math.sqrt(d) for x in kv]
        for j in range(n):
            logits[-1][:, j, :, max(0, tails[i] - n + 1 + j) :] = -math.inf
        values = [x[:, :, 1] for x in kv]
        sums = [torch.logsumexp(x, -1) if x.shape[-1] else x.new_full(x.shape[:-1], -math.inf) for x in logits]
        if s["prior"] is not None:
            sums.append(s["prior"][1][at : at + n].double().view(n, h, g).transpose(0, 1))
        whole = torch.logsumexp(torch.stack(sums), 0)
        safe = torch.where(whole == -math.inf, torch.zeros_like(whole), whole)
        o = sum(torch.einsum("hngm,hmd->nhgd", torch.exp(x - safe[..., None]), v) for x, v in zip(logits, values))
        if s["prior"] is not None:
            o = o + torch.exp(sums[-1] - safe).transpose(0, 1)[..., None] * s["prior"][0][at : at + n].double().view(n, h, g, d)
        out[at : at + n] = o.reshape(n, h * g, d)
        lse[at : at + n] = whole.transpose(0, 1).reshape(n, h * g)
        at += n
    return out, lse
