"""Cases of the operators around a request's way into the target's cache: pages for the sequences' lengths with a slot and a
position for every new token, rotary positions of queries and keys, and the attention of whole prompts over their own keys.

Pages: sequence b holds the first held[b] entries of its page_table row; `free` is a stack of free pages with `count` entries.
Lengths say how many pages each sequence shall hold: what it holds beyond them goes back, what it lacks is taken.
New tokens of sequence b are the rows start[b] .. start[b + 1] - 1, in positions ctx[b] and on (a tree's: ctx[b] + depth)."""
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
NO_PAGE = 2048  # the flag of a sequence that got no pages


def listed():
    a = dict(op="assign", page=64, ragged=True, tree=False, short=False, deepest=1)
    r = dict(op="rope", dtype="bf16", heads=32, kv_heads=8, dim=128, turned=128, adjacent=False, axes=1, ragged=True, fused=True)
    p = dict(op="prompt", dtype="bf16", heads=32, kv_heads=8, dim=128, ragged=True, fused=True, window=0, sinks=0)
    return [
        # a decoding step of a full batch: a page for each sequence whose last one is full; most of it is latency
        dict(a, name="assign-decode", batch=64, ctx=4096, new=1, kept=1, ragged=False),
        # draft trees of 32 nodes are placed, and the pages of the nodes that verify rejected go back
        dict(a, name="assign-tree", batch=64, ctx=4096, new=32, kept=6, tree=True, deepest=5),
        # prompts of odd lengths arrive while others leave, and there are too few pages for the last of them
        dict(a, name="assign-prompt", batch=250, ctx=900, new=8191, kept=8191, page=16, short=True),
        # the new tokens of a decoding step, far into long sequences
        dict(r, name="rope-decode", batch=64, ctx=100_000, new=1, ragged=False),
        # prompts of odd lengths, slices of the fused projection's output
        dict(r, name="rope-prompt", batch=8, ctx=0, new=8191),
        # video: frames of patches with a time, a height and a width each
        dict(r, name="rope-video", batch=3, ctx=517, new=5001, axes=3, heads=28, kv_heads=4),
        # in 32 bits, the first 48 of 80 dims, neighbours turned together
        dict(r, name="rope-part-f32", dtype="f32", batch=5, ctx=4096, new=301, heads=9, kv_heads=3, dim=80, turned=48, adjacent=True),
        # a short prompt of one request: latency
        dict(p, name="prompt-one", batch=1, new=37, ragged=False),
        # a batch of short prompts of odd lengths
        dict(p, name="prompt-short", batch=16, new=836),
        # two long prompts: bound by arithmetic
        dict(p, name="prompt-long", batch=2, new=8192),
        # a model with a sliding window and first tokens that stay visible, in 32 bits
        dict(p, name="prompt-window-f32", dtype="f32", batch=3, new=4001, dim=64, heads=16, kv_heads=4, window=2048, sinks=4),
        # wide heads, seven to a kv head
        dict(p, name="prompt-wide", batch=3, new=2011, dim=256, heads=14, kv_heads=2, fused=False),
    ]


def _about(rng, low, high):
    """A whole number, its logarithm spread evenly."""
    return max(low, min(high, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    case = dict(op=rng.choice(["assign", "rope", "rope", "prompt", "prompt", "prompt"]), ragged=rng.random() < 0.7)
    if case["op"] == "assign":
        case.update(batch=_about(rng, 1, 500), page=rng.choice([16, 32, 64, 128]), ctx=rng.choice([0, _about(rng, 1, 5000)]),
                    short=rng.random() < 0.3, tree=rng.random() < 0.4)
        case.update(new=_about(rng, 1, 64) if case["tree"] else _about(rng, 1, min(8191, 1_000_000 // case["batch"])))
        case.update(deepest=rng.randint(0, 16) if case["tree"] else 1, kept=rng.randint(0, case["new"]))
        return case
    case.update(dtype=rng.choice(["bf16", "bf16", "f32"]), kv_heads=rng.choice([1, 2, 3, 4, 8]), fused=rng.random() < 0.5,
                dim=rng.choice([16, 32, 48, 64, 64, 80, 96, 112, 128, 128, 128, 160, 192, 256]))
    case.update(heads=case["kv_heads"] * rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 16]))
    if case["op"] == "rope":
        case.update(batch=_about(rng, 1, 100), ctx=rng.choice([0, _about(rng, 1, 1_000_000)]), axes=rng.choice([1, 1, 2, 3]),
                    adjacent=rng.random() < 0.4, turned=case["dim"] if rng.random() < 0.6 else 16 * rng.randint(1, case["dim"] // 16))
        most = min(8191, 8 * 8191 * 40 * 64 // (case["batch"] * (case["heads"] + case["kv_heads"]) * case["dim"]))
        case.update(new=_about(rng, 1, max(1, most)))
    else:
        case.update(batch=_about(rng, 1, 64), window=0, sinks=0)
        # a third of prompt-long's work at most
        most = int((2 ** 32 // (case["batch"] * case["heads"] * (case["dim"] // 64 + 1))) ** 0.5)
        case.update(new=_about(rng, 1, max(1, min(8192, most))))
        if rng.random() < 0.4:
            case.update(window=_about(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 130]))
    return case


def _sizes(case):
    """Each sequence's cached and new tokens; by the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    b, old, most = case["batch"], case.get("ctx", 0), case["new"]
    if not case["ragged"]:
        return [old] * b, [most] * b
    return [old] + [rng.randint(old // 8, old) for _ in range(b - 1)], [most] + [rng.randint((most + 1) // 2, most) for _ in range(b - 1)]


def _pages(case):
    """Pages that each sequence holds before the call and shall hold for its tokens, and those that are free."""
    ctx, new = _sizes(case)
    page, rng = case["page"], random.Random(case["batch"] + case["new"])
    held = [-(-c // page) for c in ctx]
    # some sequences still hold pages of tokens that were not kept
    held = [h + (rng.randint(0, 3) if rng.random() < 0.2 else 0) for h in held]
    want = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    lack = sum(max(0, w - h) for w, h in zip(want, held))
    return held, want, max(1, lack * 9 // 10) if case["short"] else lack + 7


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    ctx, new = _sizes(case)
    device = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s = dict(case=case, ctx=device(ctx), most=max(new), total=starts[-1], start=device(starts) if case["ragged"] else None)
    lead = (starts[-1],) if case["ragged"] else (case["batch"], case["new"])
    if case["op"] == "assign":
        held, want, free = _pages(case)
        ids = list(range(sum(held) + free))
        rng.shuffle(ids)
        rows = []
        for h, w in zip(held, want):
            rows.append(ids[:h] + [0] * (max(map(max, held, want)) + 1 - h))
            ids = ids[h:]
        s.update(page_table=device(rows), held=device(held), pool={"free": device(ids + [0] * sum(held)), "count": device([free])},
                 status=device([0] * case["batch"]), parents=None)
        if case["tree"]:
            parents = []
            for n in new:
                depth = [0]
                parents.append(-1)
                for i in range(1, n):
                    up = rng.choice([j for j in range(max(0, i - 9), i) if depth[j] < case["deepest"]] or [0])
                    depth.append(depth[up] + 1)
                    parents.append(up)
            s["parents"] = device(parents).reshape(lead)
        # the lengths that stay: finished sequences leave, the others keep up to `kept` of the new tokens
        s["after"] = device([0 if rng.random() < 0.05 else c + rng.randint(min(n, case["kept"]) // 2, min(n, case["kept"])) for c, n in zip(ctx, new)])
        return s
    t, hq, hk, d = TYPES[case["dtype"]], case["heads"], case["kv_heads"], case["dim"]
    if case["fused"]:  # slices of one projection's output
        every = torch.randn(*lead, hq + 2 * hk, d, generator=g, device="cuda").mul_(1.2).to(t)
        s["q"], s["k"], s["v"] = every[..., :hq, :], every[..., hq:hq + hk, :], every[..., hq + hk:, :]
    else:
        s["q"], s["k"], s["v"] = (torch.randn(*lead, h, d, generator=g, device="cuda").mul_(1.2).to(t) for h in (hq, hk, hk))
    if case["op"] == "rope":
        half = case["turned"] // 2
        s["inv_freq"] = (500_000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
        first = [rng.randint(0, c) for c in ctx]
        along = [[f + i for f, n in zip(first, new) for i in range(n)]]
        if case["axes"] > 1:  # frames of 18 x 26 patches
            along = [[f + i // 468 for f, n in zip(first, new) for i in range(n)]]
            along.append([f + i % 468 // 26 for f, n in zip(first, new) for i in range(n)])
            along.append([f + i % 26 for f, n in zip(first, new) for i in range(n)])
        s["positions"] = device(along[:case["axes"]]).reshape(*((case["axes"],) if case["axes"] > 1 else ()), *lead)
        # a quarter of the pairs turn with the first axis, the others share the rest
        sections = [half] if case["axes"] == 1 else [half // 4] + [(half - half // 4) // (case["axes"] - 1)] * (case["axes"] - 1)
        sections[-1] += half - sum(sections)
        s["sections"], s["axis"] = tuple(sections), device([a for a, n in enumerate(sections) for _ in range(n)])
    return s


def run(s):
    if own:
        return _own(s)
    return {"assign": _assign, "rope": _rope, "prompt": _prompt}[s["case"]["op"]](s)


def _own(s):
    import draft_token_verification_sv_gb300 as sv
    case = s["case"]
    if case["op"] == "assign":
        got = sv.kv_assign(s["pool"], s["page_table"], s["held"], s["ctx"], case["page"], new_start=s["start"], max_new=s["most"],
                           total=s["total"] if case["ragged"] else None, parents=s["parents"], row_status=s["status"])
        status = s["status"].clone()
        sv.kv_assign(s["pool"], s["page_table"], s["held"], s["after"], case["page"])
        return dict(got, status=status, **_places(s))
    if case["op"] == "rope":
        q, k = sv.rope(s["q"], s["k"], s["positions"], s["inv_freq"], sections=s["sections"], adjacent=case["adjacent"])
        return {"q": q, "k": k}
    out, lse = sv.prompt_attention(s["q"], s["k"], s["v"], new_start=s["start"], max_new=s["most"] if case["ragged"] else None,
                                   window=case["window"], sinks=case["sinks"], lse=True)
    return {"out": out, "lse": lse}


def _places(s):
    return {"page_table": s["page_table"], "held": s["held"], "free": s["pool"]["free"], "count": s["pool"]["count"]}


# ---- the plain forms: elementary operations in 32 bits (angles in 64) ----

def _rows(s):
    """Of each new token in the order of the rows: its sequence and its place among the sequence's new ones."""
    at = torch.arange(s["total"], device="cuda")
    if s["start"] is None:
        return at // s["most"], at % s["most"]
    seq = torch.searchsorted(s["start"][1:].long(), at, right=True)
    return seq, at - s["start"].long()[seq]


def _resize(s, length):
    """Every sequence holds the pages of its length: what is over goes onto the stack, last page first, so that the first page
    given is the first one taken; sequences are served in their order while there are enough.  Says who was not."""
    table, held, free, count = s["page_table"].long(), s["held"].long(), s["pool"]["free"], s["pool"]["count"].long()
    size, page = free.shape[0], s["case"]["page"]
    want = (length + page - 1) // page
    column = torch.arange(table.shape[1], device="cuda")
    over = (column >= want[:, None]) & (column < held[:, None])
    there = count + over.sum()
    to = torch.where(over.flatten(), there - over.flatten().cumsum(0), size)
    stack = torch.cat([free, free.new_zeros(1)]).scatter(0, to, table.flatten().int())[:size]
    lack = (want - held).clamp_min(0)
    refused = (lack > 0) & (lack.cumsum(0) > there)
    holds = torch.where(refused, held, want)
    gets = (column >= held[:, None]) & (column < holds[:, None])
    at = (there - gets.flatten().cumsum(0)).clamp(0, size - 1).reshape(gets.shape)
    s["page_table"].copy_(torch.where(gets, stack[at].long(), table))
    s["held"].copy_(holds)
    free.copy_(stack)
    s["pool"]["count"].copy_(there - gets.sum())
    return refused


def _closure(reach, steps):
    return reach if steps == 0 else _closure(((reach @ reach) > 0).float(), steps - 1)


def _assign(s):
    case, page = s["case"], s["case"]["page"]
    ctx, (seq, i) = s["ctx"].long(), _rows(s)
    count = s["most"] if s["start"] is None else s["start"].long().diff()
    refused = _resize(s, ctx + count)
    place = ctx[seq] + i
    slots = s["page_table"].long()[seq, place // page] * page + place % page
    if s["parents"] is not None:  # a node's depth: how many nodes lead to it
        n = s["most"]
        parent = torch.full((case["batch"], n), -1, device="cuda")
        parent[seq, i] = s["parents"].flatten().long()
        node = torch.arange(n, device="cuda")
        reach = _closure(((parent[:, :, None] == node) | (node[:, None] == node)).float(), max(1, n - 1).bit_length())
        depth = ((reach > 0).sum(-1) - 1)[seq, i]
    else:
        depth = i
    shape = (s["total"],) if s["start"] is not None else (case["batch"], s["most"])
    got = {"slots": torch.where(refused[seq], -1, slots).reshape(shape), "positions": (ctx[seq] + depth).int().reshape(shape),
           "status": torch.where(refused, NO_PAGE, 0).int()}
    _resize(s, s["after"].long())
    return dict(got, **_places(s))


def _rope(s):
    case, half = s["case"], s["case"]["turned"] // 2
    positions = s["positions"].double().reshape(case["axes"], *s["q"].shape[:-2])
    angle = torch.movedim(positions[s["axis"]], 0, -1) * s["inv_freq"].double()
    cos, sin = angle.cos().float()[..., None, :], angle.sin().float()[..., None, :]

    def turn(x):
        y = x.float()
        a, b = (y[..., :2 * half:2], y[..., 1:2 * half:2]) if case["adjacent"] else (y[..., :half], y[..., half:2 * half])
        u, v = a * cos - b * sin, a * sin + b * cos
        turned = torch.stack((u, v), -1).flatten(-2) if case["adjacent"] else torch.cat((u, v), -1)
        return torch.cat((turned, y[..., 2 * half:]), -1).to(x.dtype)
    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _prompt(s):
    case = s["case"]
    b, hk, group, d, n = case["batch"], case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"], s["most"]
    if s["start"] is not None:  # as [B, n]: a sequence with fewer repeats its last row
        start = s["start"].long()
        row = start[:-1, None] + torch.minimum(torch.arange(n, device="cuda"), start.diff()[:, None] - 1)
    else:
        row = torch.arange(b * n, device="cuda").reshape(b, n)
    q = s["q"].reshape(-1, hk * group, d)[row].float().reshape(b, n, hk, group, d).permute(0, 2, 3, 1, 4)
    k, v = (s[x].reshape(-1, hk, d)[row].float().transpose(1, 2)[:, :, None] for x in ("k", "v"))
    i = torch.arange(n, device="cuda")
    seen = i <= i[:, None]
    if case["window"]:
        seen = seen & ((i[:, None] - i < case["window"]) | (i < case["sinks"]))
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(d ** -0.5).masked_fill_(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight, v) / total
    out = out.permute(0, 3, 1, 2, 4).reshape(b, n, hk * group, d)
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(b, n, hk * group)
    if s["start"] is not None:
        seq, at = _rows(s)
        out, lse = out[seq, at], lse[seq, at]
    return {"out": out.to(TYPES[case["dtype"]]), "lse": lse}


# ---- the operators' definitions in 64 bits ----

def exact(case, seed):
    if case["op"] == "assign":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "rope":
        half, lead, made = case["turned"] // 2, s["q"].shape[:-2], {}
        positions = s["positions"].reshape(case["axes"], *lead).double()
        parts, first = [], 0
        for a, n in enumerate(s["sections"]):  # a pair is a complex number, multiplied by exp(i angle)
            parts.append(positions[a][..., None] * s["inv_freq"][first:first + n].double())
            first += n
        by = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.cat(parts, -1))[..., None, :]
        for name in ("q", "k"):
            x = s[name].double()
            pairs = x[..., :2 * half].unflatten(-1, (half, 2)) if case["adjacent"] else x[..., :2 * half].unflatten(-1, (2, half)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by)
            made[name] = torch.cat([z.flatten(-2) if case["adjacent"] else z.transpose(-1, -2).flatten(-2), x[..., 2 * half:]], -1)
        return made
    _, new = _sizes(case)
    q, k, v = (s[x].reshape(-1, *s[x].shape[-2:]) for x in ("q", "k", "v"))
    outs, sums, first, group = [], [], 0, case["heads"] // case["kv_heads"]
    for n in new:
        rows = slice(first, first + n)
        first += n
        out = torch.empty(n, case["heads"], case["dim"], dtype=torch.float64, device="cuda")
        lse = torch.empty(n, case["heads"], dtype=torch.float64, device="cuda")
        sees = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        if case["window"]:
            sees &= sees.triu(1 - case["window"]) | (torch.arange(n, device="cuda") < case["sinks"])
        for h in range(case["heads"]):
            x = torch.einsum("id,jd->ij", q[rows, h].double(), k[rows, h // group].double()) / case["dim"] ** 0.5
            x = x.where(sees, -torch.inf)
            lse[:, h] = torch.logsumexp(x, -1)
            out[:, h] = torch.softmax(x, -1) @ v[rows, h // group].double()
        outs.append(out)
        sums.append(lse)
    join = torch.cat if case["ragged"] else torch.stack
    return {"out": join(outs), "lse": join(sums)}


def work(case):
    ctx, new = _sizes(case)
    if case["op"] == "assign":
        held, want, free = _pages(case)
        moved = sum(abs(w - h) for w, h in zip(want, held))
        # lengths, starts, held and flags of a sequence twice; a page id read and written where a page moves, there and back;
        # of a token the page id of its slot, the slot, the position and the parent
        return {"bytes": 40 * case["batch"] + 16 * moved + sum(new) * (12 + 4 / case["page"] + 4 * case["tree"]), "flops": 0}
    if case["op"] == "rope":
        values = sum(new) * (case["heads"] + case["kv_heads"])
        return {"bytes": 2 * values * case["dim"] * BYTES[case["dtype"]] + 4 * sum(new) * case["axes"], "flops": 3 * values * case["turned"]}
    w, sinks = case["window"], case["sinks"]
    pairs = sum(p + 1 if not w else min(p + 1, w + min(sinks, max(0, p + 1 - w))) for n in new for p in range(n))
    given = sum(new) * (2 * (case["heads"] + case["kv_heads"]) * case["dim"] * BYTES[case["dtype"]] + 4 * case["heads"])
    return {"bytes": given, "flops": 4 * case["dim"] * case["heads"] * pairs}
