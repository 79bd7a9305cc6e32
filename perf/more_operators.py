"""What is measured of the operators around attention: rotary positions, page tables made on
the GPU, and drafted tokens over the 4-bit cache.

``run`` computes one pass either in plain torch operations (``own`` false) or through
this package's public calls (``own`` true), on the inputs that ``prepare`` makes.

Operators, by the ``op`` of a case:
  rotary  queries and keys turned by the angle of their position, into [B, H, N, d]
  unturn  its gradient: dQ and dK turned back
  plan    page tables that grow and shrink with their requests, pages from a free list, and
          the slot and position of every new token
  tree    a tree of drafted tokens of each sequence attending over its paged 4-bit cache
  keep    drafted rows stored in the cache, the accepted ones moved together and read back
"""
import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 32  # channels that share a scale and a low value in the 4-bit cache
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _rotary(name, op, dtype, B, H, Hkv, N, d, dims, interleaved, base=10000.0, scaling="none", factor=1.0, fused=False, far=0):
    return dict(name=name, op=op, dtype=dtype, B=B, H=H, Hkv=Hkv, N=N, d=d, dims=dims, interleaved=interleaved, base=base,
                scaling=scaling, factor=factor, fused=fused, far=far)


def _plan(name, B, N, longest, page, new, done, drafts=False, spare=1.0):
    return dict(name=name, op="plan", B=B, N=N, longest=longest, page=page, new=new, done=done, drafts=drafts, spare=spare)


def _cache(name, op, dtype, B, H, Hkv, N, longest, d, page, cap=0.0, bias=False):
    return dict(name=name, op=op, dtype=dtype, B=B, H=H, Hkv=Hkv, N=N, longest=longest, d=d, page=page, cap=cap, bias=bias)


def listed():
    return [
        # one decoding step of a busy server, positions far apart: latency counts
        _rotary("rotary step", "rotary", "bf16", 64, 32, 8, 1, 128, 128, False, base=500000.0, far=131072),
        # the long training shape of the benchmark, out of a joint projection [B, N, heads, d]
        _rotary("rotary training", "rotary", "bf16", 2, 16, 4, 8192, 128, 128, False, fused=True),
        # gradients of the training shape of the benchmark, into the gradient of a joint projection, neighbouring pairs
        _rotary("unturn training", "unturn", "fp16", 4, 16, 16, 2048, 64, 64, True, fused=True),
        # gradients of a fine-tuning batch on odd pieces of long texts: wide heads, a part of the head, scaled by bands of wavelengths
        _rotary("unturn wide", "unturn", "bf16", 2, 8, 4, 2001, 256, 64, False, base=500000.0, scaling="bands", factor=8.0, far=100000),
        # one decoding step of a busy server: few sequences need a page
        _plan("plan step", 256, 1, 16384, 64, 0, 0),
        # a step with a tree of drafted tokens each, and too few pages for the last sequences
        _plan("plan drafts", 64, 24, 32768, 16, 0, 3, drafts=True, spare=0.5),
        # admission: half of the batch are new prompts, some sequences have ended
        _plan("plan prompts", 64, 8192, 16384, 16, 32, 12),
        # one short chat with a small tree: latency counts
        _cache("tree one short", "tree", "fp16", 1, 32, 8, 12, 517, 128, 16, cap=50.0),
        # a step of a busy server: 16 drafted tokens over ragged contexts
        _cache("tree batch", "tree", "bf16", 32, 32, 8, 16, 16384, 128, 64),
        # long documents, a wide tree, wide heads, a distance bias
        _cache("tree long", "tree", "bf16", 2, 16, 4, 37, 100003, 256, 128, bias=True),
        # the end of a busy server's drafted step
        _cache("keep step", "keep", "bf16", 64, 32, 8, 16, 2000, 128, 64),
        # wide trees of many sequences, wide heads, small pages
        _cache("keep wide", "keep", "fp16", 120, 16, 4, 61, 1500, 256, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes spread over the ranges, then halved until it costs no more than the largest listed one."""
    c = _drawn(rng)
    while _cost(c) > 1.0:
        if c["op"] in ("rotary", "unturn", "plan"):
            c["N"] = c["N"] // 2 + 1
        if c["op"] == "plan":
            c["B"] = c["B"] // 2 + 1
            c["new"], c["done"] = min(c["new"], c["B"] // 2), min(c["done"], c["B"] // 4)
        if c["op"] in ("tree", "keep"):
            c["B"] = max(1, c["B"] // 2)
            c["longest"] = c["longest"] // 2 + 1 if c["op"] == "tree" else c["longest"]
    return c


def _cost(c):
    """Against the largest listed case of its operator: bytes, and for trees products too."""
    w = work(c)
    if c["op"] == "tree":
        return max(w["bytes"] / 4.1e8, w["flops"] / 1e11, c["B"] * c["Hkv"] * c["longest"] * c["d"] / 6e8)
    return w["bytes"] / {"rotary": 1.7e8, "unturn": 1.7e8, "plan": 7e6, "keep": 4e7}[c["op"]]


def _drawn(rng):
    op = rng.choice(["rotary", "rotary", "unturn", "unturn", "plan", "plan", "tree", "tree", "tree", "keep"])
    if op == "plan":
        B = _log(rng, 1, 512)
        drafts = rng.random() < 0.4
        N = rng.randint(2, 64) if drafts else rng.choice([1, 1, _log(rng, 2, 8192)])
        c = _plan("", B, N, max(N, _log(rng, 64, 32768)), rng.choice([16, 32, 64, 128]), rng.randint(0, B // 2) if N > 64 else 0,
                  rng.randint(0, B // 4), drafts, rng.choice([0.3, 1.0, 1.0]))
        return {k: v for k, v in c.items() if k != "name"}
    dtype, d = rng.choice(["fp16", "bf16"]), rng.choice([64, 128, 256])
    Hkv, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 8])
    if op in ("rotary", "unturn"):
        c = _rotary("", op, dtype, _log(rng, 1, 64), Hkv * group, Hkv, rng.choice([1, _log(rng, 1, 8192), _log(rng, 1, 8192)]), d,
                    rng.choice([d, d, d // 2, d // 4]), rng.random() < 0.4, rng.choice([10000.0, 500000.0]),
                    *rng.choice([("none", 1.0), ("linear", 4.0), ("ntk", 4.0), ("bands", 8.0)]), rng.random() < 0.5, rng.choice([0, 100000]))
    elif op == "keep":
        c = _cache("", op, dtype, _log(rng, 1, 256), Hkv * group, Hkv, rng.randint(1, 64), _log(rng, 100, 4000), d, rng.choice([16, 32, 64, 128]))
    else:
        B = _log(rng, 1, 48)
        c = _cache("", op, dtype, B, Hkv * group, Hkv, rng.choice([4, 8, 16, rng.randint(1, 64), rng.randint(1, 64)]),
                   _log(rng, 70, max(80, min(60000, 500000 // B))), d, rng.choice([16, 32, 64, 128]), rng.choice([0.0, 20.0, 50.0]), rng.random() < 0.5)
    return {k: v for k, v in c.items() if k != "name"}


# ------------------------------------------------------------------------------------------ inputs


def _freqs(c):
    """Radians that each pair of channels turns by from one position to the next."""
    n, base = c["dims"], c["base"]
    if c["scaling"] == "ntk":  # a wider base: the slowest pair slows down by the factor
        base *= c["factor"] ** (n / (n - 2))
    out = []
    for i in range(n // 2):
        f = base ** (-2.0 * i / n)
        if c["scaling"] == "linear":
            f /= c["factor"]
        elif c["scaling"] == "bands":  # pairs with under 1 turn in the 8192 trained positions slow down, those with over 4 do not
            turns = 8192 * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / 3.0))
            f = f * keep + f / c["factor"] * (1.0 - keep)
        out.append(f)
    return out


def _amplitude(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "bands" else 1.0


def _lengths(c):
    """Tokens each sequence has in the cache with its draft (they depend on the case alone): the first the longest."""
    r = random.Random(c["longest"])
    lo = max(1, c["longest"] // 8, min(c["longest"], c["N"]))
    return [c["longest"]] + [r.randint(lo, c["longest"]) for _ in range(c["B"] - 1)]


def _counts(c):
    """Drafted tokens of each sequence, at most N and at most its length: the first has the most."""
    r = random.Random(c["N"] + c["longest"])
    return [min(n, c["N"] if b == 0 else r.randint(max(1, c["N"] // 2), c["N"])) for b, n in enumerate(_lengths(c))]


def _requests(c):
    """(held pages, start, count) of each sequence of a plan: the first `done` have ended, the last `new` are prompts."""
    r = random.Random(c["longest"] + c["B"])
    out = []
    for b in range(c["B"]):
        n = r.randint(max(1, c["longest"] // 8), c["longest"]) - c["N"] if c["N"] < c["longest"] else 0
        n = max(0, n)
        if b < c["done"]:
            out.append((-(-n // c["page"]), 0, 0))
        elif b >= c["B"] - c["new"]:
            out.append((0, 0, r.randint(max(1, c["N"] // 4), c["N"])))
        else:
            out.append((-(-n // c["page"]), n, min(r.randint(1, c["N"]) if c["drafts"] or not c["new"] else 1, c["longest"] - n)))
    return out


def _trees(gen, B, N):
    """Parents of drafted tokens: mostly one of the few before, -1 for children of the cached prefix."""
    i = torch.arange(N, device=DEV)
    back = 1 + (5 * torch.rand(B, N, generator=gen, device=DEV) ** 2).long()
    p = torch.clamp(i - back, min=-1)
    again = torch.rand(B, N, generator=gen, device=DEV) < 0.1
    return torch.where(again, torch.full_like(p, -1), p).to(torch.int32)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _heads(x, c):
    """Queries and keys of a joint projection [B, N, H + 2 H_kv, d], seen as [B, H, N, d]."""
    return x[:, :, : c["H"]].transpose(1, 2), x[:, :, c["H"] : c["H"] + c["Hkv"]].transpose(1, 2)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"c": c}
    if c["op"] in ("rotary", "unturn"):
        t = TYPES[c["dtype"]]
        s["freqs"] = torch.tensor(_freqs(c), dtype=torch.float64, device=DEV)
        first = torch.randint(0, c["far"] + 1, (c["B"], 1), generator=gen, device=DEV)
        s["positions"] = (first + torch.arange(c["N"], device=DEV)).to(torch.int32)
        joint = (c["B"], c["N"], c["H"] + 2 * c["Hkv"], c["d"])
        if c["fused"] and c["op"] == "rotary":
            s["q"], s["k"] = _heads(_randn(gen, *joint).to(t), c)
        else:
            s["q"] = _randn(gen, c["B"], c["H"], c["N"], c["d"]).to(t)
            s["k"] = _randn(gen, c["B"], c["Hkv"], c["N"], c["d"]).to(t)
        # the gradient of a joint projection has room for dQ, dK and dV
        s["out"] = _heads(torch.zeros(*joint, dtype=t, device=DEV), c) if c["fused"] and c["op"] == "unturn" else None
        return s
    if c["op"] == "plan":
        req = _requests(c)
        per = -(-c["longest"] // c["page"])
        held = torch.tensor([r[0] for r in req], device=DEV)
        need = sum(max(0, -(-(n + m) // c["page"]) - h) for h, n, m in req)
        free = int(need * c["spare"])
        pages = int(held.sum()) + max(free, 1)
        order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
        place = torch.arange(per, device=DEV)[None]
        before = torch.cumsum(held, 0)[:, None] - held[:, None]
        at = torch.clamp(before + place, max=pages - 1)
        table = torch.where(place < held[:, None], order[at], torch.full_like(order[at], -1))
        stack = torch.cat([order[int(held.sum()) :], torch.zeros(int(held.sum()), dtype=torch.int32, device=DEV)])[:pages]
        # what a server keeps of its pages, in one buffer: [pages on the free stack, held pages, the stack, the tables]
        s["sizes"] = [1, c["B"], pages, c["B"] * per]
        s["state"] = torch.cat([torch.tensor([free], dtype=torch.int32, device=DEV), held.to(torch.int32), stack, table.flatten()])
        s["start"] = torch.tensor([r[1] for r in req], dtype=torch.int32, device=DEV)
        s["count"] = torch.tensor([r[2] for r in req], dtype=torch.int32, device=DEV)
        s["parents"] = _trees(gen, c["B"], c["N"]) if c["drafts"] else None
        return s
    t = TYPES[c["dtype"]]
    lens = _lengths(c)
    per = -(-c["longest"] // c["page"])
    pages = c["B"] * per
    s["scale"] = 1.0 / math.sqrt(c["d"])
    s["table"] = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).view(c["B"], per).contiguous()
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["count"] = torch.tensor(_counts(c), dtype=torch.int32, device=DEV)
    s["start"] = s["lengths"] - s["count"]
    s["parents"] = _trees(gen, c["B"], c["N"])
    for n in "kv":
        s[n + "_codes"] = torch.randint(0, 256, (pages, c["Hkv"], c["page"], c["d"] // 2), generator=gen, device=DEV, dtype=torch.uint8)
        scale = 0.2 + 0.1 * torch.rand(pages, c["Hkv"], c["page"], c["d"] // GROUP, generator=gen, device=DEV)
        low = -7.5 * scale + 0.3 * _randn(gen, *scale.shape)
        s[n + "_params"] = torch.stack([scale, low], -1).to(t)
    if c["op"] == "keep":
        s["k"] = _randn(gen, c["B"], c["Hkv"], c["N"], c["d"]).to(t)
        s["v"] = _randn(gen, c["B"], c["Hkv"], c["N"], c["d"]).to(t)
        # the accepted path: some tokens of the draft in order, behind them the ones that were not
        s["path"] = torch.sort(torch.rand(c["B"], c["N"], generator=gen, device=DEV) + 2.0 * (torch.arange(c["N"], device=DEV) >= s["count"][:, None]), 1)[1]
        s["kept"] = (torch.rand(c["B"], generator=gen, device=DEV) * (s["count"].float() + 1)).to(torch.int32).clamp(max=c["N"])
        inside = torch.arange(c["N"], device=DEV)[None] < s["kept"][:, None]
        first = torch.sort(torch.where(inside, s["path"], torch.full_like(s["path"], c["N"])), 1)[0]
        s["path"] = torch.where(inside, first, torch.zeros_like(first)).to(torch.int32)
    else:
        h = torch.arange(1, c["H"] + 1, device=DEV, dtype=torch.float32)
        s["slopes"] = torch.exp2(-8.0 * h / c["H"]) if c["bias"] else None
        # capped models have larger scores: a wider q
        s["q"] = ((3.0 if c["cap"] else 1.0) * _randn(gen, c["B"], c["H"], c["N"], c["d"])).to(t)
    return s


# ------------------------------------------------------------------------------------------ plain forms


def _plain_turn(s, x, sign, out):
    c = s["c"]
    half = c["dims"] // 2
    # angles in 64 bits: positions go far
    angle = s["positions"].double()[:, None, :, None] * s["freqs"]
    cos, sin = (_amplitude(c) * torch.cos(angle)).float(), (sign * _amplitude(c) * torch.sin(angle)).float()
    y = x.float()
    if c["interleaved"]:
        a, b = y[..., 0 : c["dims"] : 2], y[..., 1 : c["dims"] : 2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half : c["dims"]]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    y = torch.cat([turned, y[..., c["dims"] :]], -1)
    return y.to(x.dtype) if out is None else out.copy_(y)


def _plain_rotary(s):
    sign = 1.0 if s["c"]["op"] == "rotary" else -1.0
    out = s["out"] or (None, None)
    return _plain_turn(s, s["q"], sign, out[0]), _plain_turn(s, s["k"], sign, out[1])


def _ancestors(parents, count):
    """[B, N, N]: whether token j is token i or one of its ancestors; no row for tokens behind count."""
    B, N = parents.shape
    i = torch.arange(N, device=DEV)
    see = ((parents[:, :, None] == i) | (i[:, None] == i)).float()
    for _ in range(max(1, (N - 1).bit_length())):  # paths of twice the length each time
        see = torch.clamp(torch.matmul(see, see), max=1.0)
    return (see > 0) & (i[:, None] < count[:, None, None])


def _plan_views(s, state):
    free_count, held, free, table = torch.split(state, s["sizes"])
    return free_count, held, free, table.view(s["c"]["B"], -1)


def _plain_plan(s):
    c = s["c"]
    state = s["state"].clone()
    free_count, held, free, table = _plan_views(s, state)
    per, room = table.shape[1], free.shape[0]
    start, count, had = s["start"].long(), s["count"].long(), held.long()
    want = -(-(start + count) // c["page"])
    place = torch.arange(per, device=DEV)[None]
    # pages that are given back lie on the stack in reverse order, so that a growth that is undone leaves it as it was
    back = torch.clamp(had - want, min=0)
    n = free_count.long() + back.sum()
    gone = (place >= want[:, None]) & (place < had[:, None])
    behind = torch.cumsum(back.flip(0), 0).flip(0) - back  # pages that later sequences give back
    to = free_count.long() + behind[:, None] + (had[:, None] - 1 - place)
    stack = torch.cat([free, free[:1]]).scatter(0, torch.where(gone, to, torch.full_like(to, room)).flatten(), table.flatten())[:room]
    # growth in the order of the sequences, as long as there are pages
    more = torch.where(want <= per, torch.clamp(want - had, min=0), torch.zeros_like(want))
    upto = torch.cumsum(more, 0)
    given = (want <= per) & ((more == 0) | (upto <= n))
    taken = torch.where(given, more, torch.zeros_like(more))
    new = given[:, None] & (place >= had[:, None]) & (place < want[:, None])
    top = n - 1 - (upto - more)[:, None] - (place - had[:, None])
    table.copy_(torch.where(new, stack[torch.clamp(top, 0, room - 1)], torch.where(gone, torch.full_like(table, -1), table)))
    free.copy_(stack)
    held.copy_(torch.where(given, want, had))
    free_count.copy_((n - taken.sum()).reshape(1))
    # every new token's place in the pool and in its sequence
    count = torch.where(given, count, torch.zeros_like(count))
    i = torch.arange(c["N"], device=DEV)[None]
    at = start[:, None] + i
    real = i < count[:, None]
    page = torch.gather(table, 1, torch.clamp(at // c["page"], max=per - 1)).long()
    slots = torch.where(real, page * c["page"] + at % c["page"], torch.full_like(at, -1))
    if s["parents"] is not None:
        at = start[:, None] + _ancestors(s["parents"], count).sum(-1) - 1
    positions = torch.where(real, at, torch.full_like(at, -1)).to(torch.int32)
    return count.to(torch.int32), (start + count).to(torch.int32), slots, positions, table, held, free, free_count


def _held(codes, params, where):
    """The values that cached rows stand for: codes and (scale, low) of the rows at ``where`` (page, row in it)."""
    page, row = where
    x = codes[page, :, row]                                   # [B, N, Hkv, d / 2]
    x = torch.stack([x & 15, x >> 4], -1).flatten(-2)          # channel 2 i is the low half of byte i
    p = params[page, :, row].double()                          # [B, N, Hkv, d / 32, 2]; the sum is rounded once, below
    x = x.double().unflatten(-1, (-1, GROUP)) * p[..., 0:1] + p[..., 1:2]
    return x.flatten(-2).to(params.dtype).transpose(1, 2)      # [B, Hkv, N, d]


def _places(s, first, n):
    """Page and row in it of the n tokens from ``first`` on of every sequence, and which of them it has."""
    c = s["c"]
    at = first.long()[:, None] + torch.arange(n, device=DEV)[None]
    have = at < s["lengths"][:, None]
    at = torch.where(have, at, torch.zeros_like(at))
    return (torch.gather(s["table"].long(), 1, at // c["page"]), at % c["page"]), have


def _plain_tree(s):
    c = s["c"]
    where, have = _places(s, torch.zeros_like(s["start"]), c["longest"])
    k = _held(s["k_codes"], s["k_params"], where).float()
    v = _held(s["v_codes"], s["v_params"], where).float()
    g = c["H"] // c["Hkv"]
    q = s["q"].float().view(c["B"], c["Hkv"], g, c["N"], c["d"])
    z = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).view(c["B"], c["Hkv"], g, c["N"], c["longest"]) * s["scale"]
    if c["cap"]:
        z = c["cap"] * torch.tanh(z / c["cap"])
    up = _ancestors(s["parents"], s["count"])                  # [B, N, N]
    j = torch.arange(c["longest"], device=DEV)
    inside = torch.clamp(j[None] - s["start"][:, None], 0, c["N"] - 1)[:, None].expand(-1, c["N"], -1)
    drafted = (j[None] >= s["start"][:, None]) & have
    see = torch.where(drafted[:, None], torch.gather(up, 2, inside), have[:, None])
    see = see & (torch.arange(c["N"], device=DEV)[None, :, None] < s["count"][:, None, None])
    if s["slopes"] is not None:
        depth = up.sum(-1) - 1                                 # a token's position is the prefix and its depth
        mine = s["start"][:, None] + depth
        theirs = torch.where(drafted, s["start"][:, None] + torch.gather(depth, 1, inside[:, 0]), j[None])
        away = (mine[:, :, None] - theirs[:, None]).abs().float()
        z = z - s["slopes"].view(1, c["Hkv"], g, 1, 1) * away[:, None, None]
    z = z.masked_fill_(~see[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)     # rows that see nothing
    p = torch.exp(z.sub_(m))
    l = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(l > 0, l, torch.ones_like(l)))
    lse = (m + torch.log(l))[..., 0]
    o = torch.matmul(p.flatten(2, 3), v)
    return o.reshape(s["q"].shape).to(s["q"].dtype), lse.reshape(c["B"], c["H"], c["N"])


def _coded(x):
    """Codes and (scale, low) of rows x, every step in 32 bits."""
    g = x.float().unflatten(-1, (-1, GROUP))
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale = ((high - low) / 15.0).to(x.dtype).float()
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    inv = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
    q = torch.clamp(torch.round((g - low) * inv), max=15.0).to(torch.uint8).flatten(-2)
    return q[..., 0::2] | (q[..., 1::2] << 4), torch.cat([scale, low], -1).to(x.dtype)


def _plain_keep(s):
    c = s["c"]
    (page, row), _ = _places(s, s["start"], c["N"])
    i = torch.arange(c["N"], device=DEV)[None]
    new = (i < s["count"][:, None]).nonzero(as_tuple=True)
    into = (i < s["kept"][:, None]).nonzero(as_tuple=True)
    path = s["path"].long()
    out = []
    kept = (i < s["kept"][:, None])[:, None, :, None]
    for name in "kv":
        codes, params = _coded(s[name])
        # the draft's rows, then the accepted ones behind the prefix
        for pool, x in ((s[name + "_codes"], codes), (s[name + "_params"], params)):
            pool[page[new], :, row[new]] = x.transpose(1, 2)[new]
            at = torch.gather(page, 1, path), torch.gather(row, 1, path)
            pool[page[into], :, row[into]] = pool[at[0][into], :, at[1][into]]
        out.append(_held(s[name + "_codes"], s[name + "_params"], (page, row)).masked_fill(~kept, 0.0))
    return tuple(out)


# ------------------------------------------------------------------------------------------ one pass


def run(state):
    s = state
    c = s["c"]
    if own:
        import exact_attention_37_gb300 as fa

        if c["op"] == "rotary":
            return fa.rotary(s["q"], s["k"], s["positions"], s["freqs"], interleaved=c["interleaved"], amplitude=_amplitude(c))
        if c["op"] == "unturn":
            return fa.rotary_backward(s["q"], s["k"], s["positions"], s["freqs"], interleaved=c["interleaved"], amplitude=_amplitude(c),
                                      out=s["out"])
        if c["op"] == "plan":
            free_count, held, free, table = _plan_views(s, s["state"].clone())
            new = fa.kv4_plan(fa.KV4Pages(table, held, free, free_count), c["page"], s["start"], s["count"], c["N"], parents=s["parents"])
            return (*new, table, held, free, free_count)
        cache = fa.KV4Cache(s["k_codes"], s["k_params"], s["v_codes"], s["v_params"])
        if c["op"] == "tree":
            return fa.kv4_attend_tree(s["q"], cache, s["table"], s["lengths"], s["parents"], s["count"], scale=s["scale"], cap=c["cap"],
                                      slopes=s["slopes"])
        fa.kv4_append(cache, s["k"], s["v"], s["table"], s["start"], s["count"])
        fa.kv4_keep(cache, s["table"], s["start"], s["path"], s["kept"])
        return fa.kv4_read(cache, s["table"], s["start"], c["N"], s["start"] + s["kept"])
    return {"rotary": _plain_rotary, "unturn": _plain_rotary, "plan": _plain_plan, "tree": _plain_tree, "keep": _plain_keep}[c["op"]](s)


def work(case):
    c = case
    if c["op"] in ("rotary", "unturn"):
        heads = (c["H"] + c["Hkv"]) * c["B"] * c["N"]
        return {"bytes": 2 * 2 * heads * c["d"] + 4 * c["B"] * c["N"] + 4 * c["dims"], "flops": 3 * heads * c["dims"]}
    if c["op"] == "plan":
        req = _requests(c)
        moved = sum(abs(-(-(n + m) // c["page"]) - h) for h, n, m in req)
        touched = sum(-(-m // c["page"]) for _, _, m in req)
        # requests in and out, pages between list and tables, the tables' places of new tokens, slots and positions
        return {"bytes": 24 * c["B"] + 8 * moved + 4 * touched + c["B"] * c["N"] * (16 if c["drafts"] else 12), "flops": 0}
    lens, counts = _lengths(c), _counts(c)
    row = 2 * c["Hkv"] * (c["d"] // 2 + c["d"] // GROUP * 4)  # a cached token: keys and values
    if c["op"] == "keep":
        full = 2 * c["Hkv"] * c["d"] * 2
        kept = sum(counts) // 2
        return {"bytes": sum(counts) * (full + row) + kept * (2 * row + full), "flops": 0}
    qo = c["B"] * c["H"] * c["N"] * (2 * c["d"] * 2 + 4)
    seen = sum(m * (n - m + 1) for n, m in zip(lens, counts))
    return {"bytes": sum(lens) * row + qo, "flops": 4 * c["d"] * c["H"] * seen}


# ------------------------------------------------------------------------------------------ in 64 bits


def _exact_values(s, name, b, h, n):
    """Rows 0 .. n - 1 of one cached head of one sequence, in 64 bits; the stored value is rounded to the cache's type."""
    c = s["c"]
    tok = torch.arange(n, device=DEV)
    page = s["table"][b].long()[tok // c["page"]]
    raw = s[name + "_codes"][page, h, tok % c["page"]].long()
    par = s[name + "_params"][page, h, tok % c["page"]].double()
    val = torch.empty(n, c["d"], dtype=torch.float64, device=DEV)
    for ch in range(c["d"]):
        val[:, ch] = par[:, ch // GROUP, 1] + ((raw[:, ch // 2] >> (4 * (ch % 2))) & 15) * par[:, ch // GROUP, 0]
    return val.to(TYPES[c["dtype"]]).double()


def _exact_turn(s, x, sign):
    c = s["c"]
    turns = s["positions"].double()[..., None] * (s["freqs"] / (2 * math.pi))
    angle = 2 * math.pi * (turns - torch.round(turns))
    z = torch.polar(torch.full_like(angle, _amplitude(c)), sign * angle)[:, None]
    y = x.double().clone()
    n = c["dims"]
    lo, hi = (slice(0, n, 2), slice(1, n, 2)) if c["interleaved"] else (slice(0, n // 2), slice(n // 2, n))
    w = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * z
    y[..., lo], y[..., hi] = w.real, w.imag
    return y


def exact(case, seed):
    c = case
    if c["op"] == "plan":
        return None
    s = prepare(c, seed)
    f8 = dict(dtype=torch.float64, device=DEV)
    if c["op"] in ("rotary", "unturn"):
        sign = 1.0 if c["op"] == "rotary" else -1.0
        return _exact_turn(s, s["q"], sign), _exact_turn(s, s["k"], sign)
    if c["op"] == "keep":
        # the code of a value is chosen in steps of 32 bits by definition; what it stands for is taken in 64
        outs = []
        for name in "kv":
            x = s[name].float().view(c["B"], c["Hkv"], c["N"], -1, GROUP)
            low = x.min(-1, keepdim=True)[0]
            step = ((x.max(-1, keepdim=True)[0] - low) / 15).to(TYPES[c["dtype"]]).float()
            step = step * (step >= 2.0 ** -126)
            code = torch.where(step > 0, torch.round((x - low) * (1 / step)).clamp(max=15), torch.zeros_like(x))
            vals = (low.double() + code.double() * step.double()).to(TYPES[c["dtype"]]).double().flatten(-2)
            out = torch.zeros_like(vals)
            for b in range(c["B"]):
                n = int(s["kept"][b])
                out[b, :, :n] = vals[b][:, s["path"][b, :n].long()]
            outs.append(out)
        return tuple(outs)
    o, lse = torch.zeros(s["q"].shape, **f8), torch.full(s["q"].shape[:3], -math.inf, **f8)
    parents, g = s["parents"].tolist(), c["H"] // c["Hkv"]
    for b in range(c["B"]):
        n, m = int(s["lengths"][b]), int(s["count"][b])
        see = torch.zeros(m, n, dtype=torch.bool, device=DEV)
        see[:, : n - m] = True
        depth, rows = [], []
        for i in range(m):
            p = parents[b][i]
            rows.append([i] if p < 0 else rows[p] + [i])
            depth.append(len(rows[i]) - 1)
            see[i, torch.tensor(rows[i], device=DEV) + (n - m)] = True
        pos = torch.tensor([float(n - m + x) for x in depth], **f8)
        away = (pos[:, None] - torch.cat([torch.arange(n - m, **f8), pos])[None]).abs()
        for hk in range(c["Hkv"]):
            k, v = _exact_values(s, "k", b, hk, n), _exact_values(s, "v", b, hk, n)
            for h in range(hk * g, hk * g + g):
                z = (s["q"][b, h, :m].double() @ k.t()) * float(torch.tensor(s["scale"], dtype=torch.float32))
                if c["cap"]:
                    z = c["cap"] * torch.tanh(z / c["cap"])
                if s["slopes"] is not None:
                    z = z - float(s["slopes"][h]) * away
                z[~see] = -math.inf
                lse[b, h, :m] = torch.logsumexp(z, -1)
                o[b, h, :m] = torch.exp(z - lse[b, h, :m, None]) @ v
    return o, lse
