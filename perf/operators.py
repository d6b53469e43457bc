"""Cases of the operators around a scoring pass over drafted tokens: the 8-bit cache that the target model keeps of its
context (written, read back, committed along the accepted path) and the attention of the drafted tokens over it.

A cache holds e4m3 codes in pages of `page` tokens with one power-of-two scale for each (page, kv head); a stored value is
code * scale.  Sequence b owns the pages page_table[b]; its token j lies in page page_table[b, j // page], slot j % page.
ctx[b] tokens are cached before the call; the call's new tokens follow them."""
import random

import torch

own = False

CODE = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
SMALLEST = 2.0 ** -100  # the smallest scale


def listed():
    a = dict(op="append", dtype="bf16", heads=32, kv_heads=8, dim=128, page=64, layout="hnd", fused=True, ragged=True)
    r = dict(op="read", dtype="bf16", kv_heads=8, dim=128, page=64, layout="hnd", ragged=True)
    t = dict(op="attend", dtype="bf16", heads=32, kv_heads=8, dim=128, page=64, layout="hnd", fused=False, ragged=True, tree=False, window=0, sinks=0)
    c = dict(op="commit", kv_heads=8, dim=128, page=64, layout="hnd", ragged=True)
    return [
        # each of 64 requests caches the one token of a decoding step, out of the fused projection's output
        dict(a, name="append-decode", batch=64, ctx=4096, new=1),
        # prompts of odd lengths arrive together
        dict(a, name="append-prompt", batch=8, ctx=0, new=8191, page=128, layout="nhd"),
        # a short odd stretch in 32 bits, as a test or a transfer of one request takes it
        dict(r, name="read-odd", dtype="f32", batch=3, first=5, tokens=333, kv_heads=2, dim=80, page=16),
        # two long contexts are taken out of the cache
        dict(r, name="read-long", batch=2, first=0, tokens=65537),
        # one request, one token: latency
        dict(t, name="attend-one", batch=1, ctx=500, new=1, ragged=False),
        # a decoding step of a full batch
        dict(t, name="attend-decode", batch=64, ctx=8192, new=1),
        # a chain of 7 drafted tokens and the last one, long contexts
        dict(t, name="attend-chain", batch=16, ctx=32768, new=8, fused=True),
        # draft trees of 32 nodes
        dict(t, name="attend-tree", batch=64, ctx=4096, new=32, ragged=True, tree=True),
        # a model with a sliding window and first tokens that stay visible, in 32 bits, chains of 5 drafts and fewer
        dict(t, name="attend-window-f32", dtype="f32", batch=32, ctx=20000, new=6, dim=64, heads=16, kv_heads=4, page=16, layout="nhd", window=2048, sinks=4),
        # a stretch of a prompt on top of what is cached: bound by arithmetic
        dict(t, name="attend-prompt", batch=2, ctx=4096, new=2000, page=128),
        # the accepted paths of 64 trees of 32 nodes, depth 5
        dict(c, name="commit-tree", batch=64, ctx=4096, nodes=32, depth=5),
        # larger and deeper trees, small pages
        dict(c, name="commit-deep", batch=256, ctx=700, nodes=64, depth=16, kv_heads=4, dim=64, page=16, layout="nhd"),
    ]


def _about(rng, low, high):
    """A whole number, its logarithm spread evenly."""
    return max(low, min(high, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    case = dict(op=rng.choice(["append", "read", "attend", "attend", "attend", "commit"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                kv_heads=rng.choice([1, 2, 3, 4, 8]), dim=rng.choice([32, 48, 64, 64, 80, 96, 112, 128, 128, 128, 160, 192, 256]),
                page=rng.choice([16, 32, 64, 128]), layout=rng.choice(["hnd", "nhd"]), ragged=rng.random() < 0.7)
    heads = case["kv_heads"] * rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 16])
    if case["op"] == "append":
        case.update(heads=heads, fused=rng.random() < 0.5, batch=_about(rng, 1, 200), ctx=rng.choice([0, _about(rng, 1, 5000)]))
        most = min(8191, 40_000_000 // (case["batch"] * case["kv_heads"] * case["dim"]))
        case.update(new=_about(rng, 1, max(1, most)))
    elif case["op"] == "read":
        case.update(batch=_about(rng, 1, 100), first=rng.choice([0, _about(rng, 1, 500)]))
        most = min(60000, 50_000_000 // (case["batch"] * case["kv_heads"] * case["dim"]))
        case.update(tokens=_about(rng, 1, max(1, most)))
    elif case["op"] == "commit":
        del case["dtype"]
        case.update(batch=_about(rng, 1, 256), ctx=_about(rng, 1, 3000), nodes=_about(rng, 1, 64))
        case.update(depth=rng.randint(0, min(16, case["nodes"] - 1)))
    else:
        case.update(heads=heads, fused=rng.random() < 0.5, batch=_about(rng, 1, 128), new=rng.choice([1, _about(rng, 2, 65), _about(rng, 2, 65), _about(rng, 66, 1000)]))
        case.update(tree=1 < case["new"] <= 65 and rng.random() < 0.5)
        most = min(100_000, 300_000_000 // (case["batch"] * case["kv_heads"] * case["dim"]), 150_000_000 // (case["batch"] * heads * case["new"]),
                   160_000_000_000 // (4 * case["batch"] * heads * case["new"] * case["dim"]))
        case.update(ctx=rng.choice([0] + 5 * [_about(rng, 1, max(1, most))]), window=0, sinks=0)
        if rng.random() < 0.4:
            case.update(window=_about(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 17]))
    return case


def _sizes(case):
    """Each sequence's cached and new tokens (read: the first and the number); by the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    b, old, most = case["batch"], case.get("ctx", case.get("first", 0)), case.get("new", case.get("tokens", case.get("nodes")))
    if not case["ragged"]:
        return [old] * b, [most] * b
    ctx = [old] + [rng.randint(old // 8, old) for _ in range(b - 1)]
    return ctx, [most] * b if case["op"] == "commit" else [most] + [rng.randint((most + 1) // 2, most) for _ in range(b - 1)]


def _accepted(case):
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")) + "accepted")
    return [rng.randint(0, case["depth"]) for _ in range(case["batch"])]


def _heap(g, case, pages):
    """Codes of both caches and their scales, as an earlier pass leaves them: values about N(0, 1)."""
    n, h, p, d = pages, case["kv_heads"], case["page"], case["dim"]
    made = {}
    for name in ("k", "v"):
        shape = (n, p, h, d) if case["layout"] == "nhd" else (n, h, p, d)
        codes = torch.empty(shape, dtype=CODE, device="cuda")
        for at in range(0, n, max(1, (1 << 27) // (h * p * d))):
            part = codes[at:at + max(1, (1 << 27) // (h * p * d))]
            part.copy_((torch.randn(part.shape, generator=g, device="cuda", dtype=torch.bfloat16) * 75).clamp_(-448, 448))
        made[name] = codes.transpose(1, 2) if case["layout"] == "nhd" else codes
        made[name + "_scale"] = torch.exp2(-torch.randint(5, 8, (n, h), generator=g, device="cuda").float())
    return made


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    ctx, new = _sizes(case)
    b, page = case["batch"], case["page"]
    columns = max(1, max(-(-(c + n) // page) for c, n in zip(ctx, new)))
    used = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    total = sum(used) + 3  # a few pages are free
    ids = list(range(total))
    rng.shuffle(ids)
    rows = []
    for n in used:
        rows.append(ids[:n] + [0] * (columns - n))
        ids = ids[n:]
    device = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(case=case, cache=_heap(g, case, total), page_table=device(rows), ctx=device(ctx), most=max(new), longest=max(c + n for c, n in zip(ctx, new)))
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["start"] = device(starts) if case["ragged"] and case["op"] != "commit" else None
    s["total"] = starts[-1]
    lead = (starts[-1],) if case["ragged"] else (b, case.get("new", 1))
    if case["op"] in ("append", "attend"):
        t, hq, hk, d = TYPES[case["dtype"]], case["heads"], case["kv_heads"], case["dim"]
        if case["fused"]:  # slices of one projection's output
            every = torch.randn(*lead, hq + 2 * hk, d, generator=g, device="cuda").mul_(1.2).to(t)
            s["q"], s["k"], s["v"] = every[..., :hq, :], every[..., hq:hq + hk, :], every[..., hq + hk:, :]
        elif case["op"] == "append":
            s["k"], s["v"] = (torch.randn(*lead, hk, d, generator=g, device="cuda").to(t) for _ in range(2))
        else:
            s["q"] = torch.randn(*lead, hq, d, generator=g, device="cuda").mul_(1.5).to(t)
    if case["op"] == "attend":
        s["parents"] = None
        if case["tree"]:  # a parent among the last few nodes keeps the trees deep
            parents = [[-1] + [rng.randint(max(0, i - 9), i - 1) for i in range(1, n)] for n in new]
            s["parents"] = device([x for row in parents for x in row]).reshape(lead)
    if case["op"] == "commit":
        s["accept"] = device(_accepted(case))
        paths = [[0] + sorted(rng.sample(range(1, case["nodes"]), a)) for a in _accepted(case)]
        s["path"] = device([p + [-1] * (case["depth"] + 1 - len(p)) for p in paths])
    return s


def run(s):
    case = s["case"]
    if own:
        return _own(s)
    return {"append": _append, "read": _read, "attend": _attend, "commit": _commit}[case["op"]](s)


def _own(s):
    import draft_token_verification_sv_gb300 as sv
    case, cache = s["case"], s["cache"]
    if case["op"] == "append":
        sv.kv_append(cache, s["k"], s["v"], s["page_table"], s["ctx"], new_start=s["start"], max_new=s["most"])
        return _held(cache)
    if case["op"] == "read":
        k, v = sv.kv_read(cache, s["page_table"], s["ctx"], s["most"], new_start=s["start"], total=s["total"], dtype=TYPES[case["dtype"]])
        return {"k": k, "v": v}
    if case["op"] == "commit":
        lens = sv.kv_commit(cache, s["page_table"], s["ctx"], s["path"], s["accept"], case["nodes"])
        return dict(_held(cache), lens=lens)
    out, lse = sv.kv_attention(s["q"], cache, s["page_table"], s["ctx"], new_start=s["start"], max_new=s["most"], parents=s["parents"],
                               window=case["window"], sinks=case["sinks"], lse=True)
    return {"out": out, "lse": lse}


def _held(cache):
    """What the cache holds: 8-bit values and scales."""
    return {"k": cache["k"].view(CODE), "v": cache["v"].view(CODE), "k_scale": cache["k_scale"], "v_scale": cache["v_scale"]}


# ---- the plain forms: elementary operations in 32 bits ----

def _places(s):
    """Of each new token in the order of the rows of [total, ...]: its sequence and its place among the sequence's new ones."""
    b, most = s["case"]["batch"], s["most"]
    at = torch.arange(s["total"], device="cuda")
    if s["start"] is None:
        return at // most, at % most
    seq = torch.searchsorted(s["start"][1:].long(), at, right=True)
    return seq, at - s["start"].long()[seq]


def _need(largest):
    """The smallest power of two s with largest / s <= 448."""
    m, e = torch.frexp(largest / 448.0)
    s = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))
    return torch.where(largest > 0, s, torch.zeros_like(s)).clamp_min(SMALLEST)


def _codes(x):
    return torch.nan_to_num(x, nan=0.0).clamp(-448.0, 448.0).to(CODE).view(torch.uint8)


def _store(s, name, x, seq, pos):
    """Puts x [T, kv_heads, dim] (32 bits) at positions pos of the sequences seq, each of which gets one token or more."""
    codes, scale, page, table = s["cache"][name].view(torch.uint8), s["cache"][name + "_scale"], s["case"]["page"], s["page_table"].long()
    ctx = s["ctx"].long()
    at = table[seq, pos // page]
    largest = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    top = torch.zeros_like(scale).scatter_reduce(0, at[:, None].expand_as(largest), largest, "amax")
    ones = lambda i: torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").index_fill(0, i, True)[:, None]  # noqa: E731
    touched = ones(at)
    # a page that holds earlier tokens keeps its scale or grows it, and those tokens' codes follow
    first, held = table.gather(1, (ctx // page)[:, None])[:, 0], ctx % page
    before = torch.zeros_like(scale).index_copy(0, first, torch.where(held[:, None] > 0, scale[first], 0.0))
    grown = torch.where(touched, torch.maximum(before, _need(top)), scale)
    old = codes[first]  # [B, kv_heads, page, dim]
    again = _codes(old.view(CODE).float() * (scale[first] / grown[first])[..., None, None])
    codes[first] = torch.where((torch.arange(page, device="cuda") < held[:, None])[:, None, :, None], again, old)
    codes[at, :, pos % page] = _codes(x / grown[at][..., None])
    scale.copy_(grown)


def _take(s, name, seq, pos):
    """Values [T, kv_heads, dim] (32 bits) of positions pos of the sequences seq."""
    cache, page = s["cache"], s["case"]["page"]
    at = s["page_table"].long()[seq, pos // page]
    return cache[name].view(torch.uint8)[at, :, pos % page].view(CODE).float() * cache[name + "_scale"][at][..., None]


def _append(s):
    seq, i = _places(s)
    for_each = s["ctx"].long()[seq] + i
    _store(s, "k", s["k"].reshape(s["total"], *s["k"].shape[-2:]).float(), seq, for_each)
    _store(s, "v", s["v"].reshape(s["total"], *s["v"].shape[-2:]).float(), seq, for_each)
    return _held(s["cache"])


def _read(s):
    seq, i = _places(s)
    pos, t = s["ctx"].long()[seq] + i, TYPES[s["case"]["dtype"]]
    shape = (s["total"],) if s["start"] is not None else (s["case"]["batch"], s["most"])
    return {n: _take(s, n, seq, pos).to(t).reshape(*shape, s["case"]["kv_heads"], s["case"]["dim"]) for n in ("k", "v")}


def _commit(s):
    b, deep = s["path"].shape
    # what lies past the accepted node repeats the path's first node
    i = torch.arange(deep, device="cuda").expand(b, deep)
    i = torch.where(i <= s["accept"].long()[:, None], i, 0).reshape(-1)
    seq = torch.arange(b, device="cuda").repeat_interleave(deep)
    ctx = s["ctx"].long()[seq]
    node = s["path"].long()[seq, i]
    kept = {n: _take(s, n, seq, ctx + node) for n in ("k", "v")}
    _store(s, "k", kept["k"], seq, ctx + i)
    _store(s, "v", kept["v"], seq, ctx + i)
    return dict(_held(s["cache"]), lens=s["ctx"] + s["accept"] + 1)


def _closure(reach, steps):
    return reach if steps == 0 else _closure(((reach @ reach) > 0).float(), steps - 1)


def _attend(s):
    case, page = s["case"], s["case"]["page"]
    b, hk, group, d, n, length = case["batch"], case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"], s["most"], s["longest"]
    ctx, ragged = s["ctx"].long(), s["start"] is not None
    # queries and parents as [B, n]: a sequence with fewer repeats its last one
    if ragged:
        start = s["start"].long()
        count = start[1:] - start[:-1]
        row = start[:-1, None] + torch.minimum(torch.arange(n, device="cuda"), count[:, None] - 1)
    else:
        row = torch.arange(b * n, device="cuda").reshape(b, n)
    q = s["q"].reshape(-1, hk * group, d)[row].float().reshape(b, n, hk, group, d).permute(0, 2, 1, 3, 4).reshape(b, hk, n * group, d)
    pages = s["page_table"].long()[:, : -(-length // page)]
    values = lambda name: (s["cache"][name].view(torch.uint8)[pages].view(CODE).float() * s["cache"][name + "_scale"][pages][..., None, None]).transpose(1, 2).reshape(b, hk, -1, d)[:, :, :length]  # noqa: E731
    j, i = torch.arange(length, device="cuda"), torch.arange(n, device="cuda")
    if s["parents"] is not None:
        parent = s["parents"].reshape(-1).long()[row]
        edge = (parent[:, :, None] == i) & (i[:, None] > i)
        reach = _closure((edge | (i[:, None] == i)).float(), max(1, n - 1).bit_length()) > 0
        depth = reach.sum(-1) - 1
        new = j - ctx[:, None]  # [B, length]
        here = new.clamp(0, n - 1)
        seen = (new < 0)[:, None] | (reach.gather(2, here[:, None].expand(b, n, length)) & (new < n)[:, None])
        at = torch.where(new < 0, j, ctx[:, None] + depth.gather(1, here))
        mine = ctx[:, None] + depth
    else:
        mine = ctx[:, None] + i
        seen, at = j <= mine[:, :, None], j.expand(b, length)
    if case["window"]:
        seen = seen & ((mine[:, :, None] - at[:, None] < case["window"]) | (at < case["sinks"])[:, None])
    seen = seen[:, None, :, None].expand(b, 1, n, group, length).reshape(b, 1, n * group, length)
    score = (q @ values("k").transpose(2, 3)) * d ** -0.5
    score = score.masked_fill_(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    weight = torch.exp_(score.sub_(torch.where(top.isfinite(), top, 0.0)))
    total = weight.sum(-1, keepdim=True)
    out = (weight @ values("v")) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log())[..., 0]
    out = out.reshape(b, hk, n, group, d).permute(0, 2, 1, 3, 4).reshape(b, n, hk * group, d)
    lse = lse.reshape(b, hk, n, group).permute(0, 2, 1, 3).reshape(b, n, hk * group)
    if ragged:
        seq, k = _places(s)
        out, lse = out[seq, k], lse[seq, k]
    return {"out": out.to(TYPES[case["dtype"]]), "lse": lse}


# ---- the operators' definitions in 64 bits ----

def _value64(cache, name, page, slots):
    return cache[name][page][:, slots].double() * cache[name + "_scale"][page].double()[:, None, None]


def _sequence64(s, name, seq, first, last):
    """Tokens [first, last) of a sequence: [kv_heads, tokens, dim]."""
    page, table = s["case"]["page"], s["page_table"][seq].tolist()
    parts = [_value64(s["cache"], name, table[g], slice(max(first, g * page) - g * page, min(last, (g + 1) * page) - g * page)) for g in range(first // page, -(-last // page))]
    return torch.cat(parts, 1)


def _rounded64(x):
    """The nearest value that e4m3 has, ties to even."""
    x = x.clamp(-448, 448)
    power = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -20))).clamp_min(-6)
    step = torch.exp2(power - 3)
    return torch.round(x / step) * step


def _scale64(largest):
    """By trial: the powers of two about largest / 448."""
    guess = torch.round(torch.log2(largest.clamp_min(2.0 ** -300) / 448))
    fits = lambda e: largest <= 448 * torch.exp2(e)  # noqa: E731
    e = torch.where(fits(guess - 1), guess - 1, torch.where(fits(guess), guess, guess + 1))
    return torch.exp2(e.clamp_min(-100))


def _stored64(s, made, name, seq, first, x):
    """Tokens first.. of a sequence become x [tokens, kv_heads, dim]; `made`: the values of the codes and the scales."""
    page, table, codes, scale = s["case"]["page"], s["page_table"][seq].tolist(), made[name], made[name + "_scale"]
    last = first + x.shape[0]
    for g in range(first // page, -(-last // page)):
        lo, hi, at = max(first, g * page), min(last, (g + 1) * page), table[g]
        part = x[lo - first:hi - first]
        new = _scale64(part.abs().amax((0, 2)))
        held = max(0, first - g * page)
        if held:
            new = torch.maximum(new, scale[at])
            codes[at, :, :held] = _rounded64(codes[at, :, :held] * (scale[at] / new)[:, None, None])
        codes[at, :, lo - g * page:hi - g * page] = _rounded64(part / new[None, :, None]).transpose(0, 1)
        scale[at] = new


def exact(case, seed):
    s = prepare(case, seed)
    ctx, new = _sizes(case)
    starts = [sum(new[:k]) for k in range(len(new))]
    if case["op"] in ("append", "commit"):
        made = {n: t.double() for n, t in s["cache"].items()}
        for seq, first in enumerate(ctx):
            if case["op"] == "append":
                given = {n: s[n].reshape(-1, *s[n].shape[-2:])[starts[seq]:starts[seq] + new[seq]].double() for n in ("k", "v")}
            else:
                nodes = s["path"][seq].tolist()[: _accepted(case)[seq] + 1]
                given = {n: _sequence64(s, n, seq, first, first + case["nodes"]).transpose(0, 1)[nodes] for n in ("k", "v")}
            for n in ("k", "v"):
                _stored64(s, made, n, seq, first, given[n])
        return made if case["op"] == "append" else dict(made, lens=None)
    if case["op"] == "read":
        parts = {n: [_sequence64(s, n, q, c, c + m).transpose(0, 1) for q, (c, m) in enumerate(zip(ctx, new))] for n in ("k", "v")}
        return {n: torch.cat(p) if case["ragged"] else torch.stack(p) for n, p in parts.items()}
    q, outs, sums = s["q"].reshape(-1, *s["q"].shape[-2:]).double(), [], []
    for seq, (c, m) in enumerate(zip(ctx, new)):
        k, v = (_sequence64(s, n, seq, 0, c + m) for n in ("k", "v"))
        depth, sees = list(range(m)), torch.zeros(m, m, dtype=torch.bool)
        if case["tree"]:
            parent = s["parents"].reshape(-1)[starts[seq]:starts[seq] + m].tolist()
            for i, p in enumerate(parent):
                depth[i] = 0 if p < 0 else depth[p] + 1
                if p >= 0:
                    sees[i] = sees[p]
                sees[i, i] = True
        else:
            sees = torch.ones(m, m, dtype=torch.bool).tril()
        place = torch.tensor(list(range(c)) + [c + x for x in depth], device="cuda")
        sees = torch.cat([torch.ones(m, c, dtype=torch.bool), sees], 1).cuda()
        if case["window"]:
            sees &= (place[c:, None] - place < case["window"]) | (place < case["sinks"])
        mine = q[starts[seq]:starts[seq] + m].reshape(m, case["kv_heads"], -1, case["dim"])
        out, lse = [], []
        for h in range(case["kv_heads"]):
            x = torch.einsum("ngd,ld->ngl", mine[:, h], k[h]) / case["dim"] ** 0.5
            x = x.masked_fill(~sees[:, None], -float("inf"))
            lse.append(torch.logsumexp(x, -1))
            out.append(torch.einsum("ngl,ld->ngd", torch.softmax(x, -1), v[h]))
        outs.append(torch.stack(out, 1).reshape(m, case["heads"], case["dim"]))
        sums.append(torch.stack(lse, 1).reshape(m, case["heads"]))
    join = torch.cat if case["ragged"] else torch.stack
    return {"out": join(outs), "lse": join(sums)}


def _pairs(case, ctx, new):
    """Visible (query, token) pairs of a sequence, and the tokens that any query sees; a tree's nodes count as a chain's."""
    w, sinks = case["window"], case["sinks"]
    pairs = sum(p + 1 if not w else min(p + 1, w + min(sinks, max(0, p + 1 - w))) for p in range(ctx, ctx + new))
    tokens = ctx + new if not w else min(ctx + new, w + new - 1 + min(sinks, max(0, ctx + 1 - w)))
    return pairs, tokens


def work(case):
    ctx, new = _sizes(case)
    row = case["kv_heads"] * case["dim"]  # values of a token in one of the caches
    pages = lambda first, last: -(-last // case["page"]) - first // case["page"]  # noqa: E731
    if case["op"] == "append":
        scales = sum(pages(c, c + m) for c, m in zip(ctx, new)) * case["kv_heads"] * 4
        return {"bytes": 2 * (sum(new) * row * (BYTES[case["dtype"]] + 1) + scales), "flops": 0}
    if case["op"] == "read":
        scales = sum(pages(c, c + m) for c, m in zip(ctx, new)) * case["kv_heads"] * 4
        return {"bytes": 2 * (sum(new) * row * (BYTES[case["dtype"]] + 1) + scales), "flops": 0}
    if case["op"] == "commit":
        kept = sum(_accepted(case)) + case["batch"]
        return {"bytes": 2 * (2 * kept * row + kept * case["kv_heads"] * 4), "flops": 0}
    each = [_pairs(case, c, m) for c, m in zip(ctx, new)]
    tokens = sum(t for _, t in each)
    given = sum(new) * case["heads"] * (2 * case["dim"] * BYTES[case["dtype"]] + 4)
    return {"bytes": 2 * tokens * row + 2 * -(-tokens // case["page"]) * case["kv_heads"] * 4 + given, "flops": 4 * case["dim"] * case["heads"] * sum(p for p, _ in each)}
