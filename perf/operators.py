"""What is measured of the attention operators that work on changed scores and on a 4-bit cache.

``run`` computes one pass either in plain torch operations (``own`` false) or through
this package's public calls (``own`` true), on the inputs that ``prepare`` makes.

Operators, by the ``op`` of a case:
  fwd     attention with a score rule: tanh cap, distance bias, document ids, prefix, causal
  bwd     its gradients dQ, dK, dV from O, L and dO
  store   new key/value rows into a paged 4-bit cache, then the rows the cache holds read back
  attend  a few new tokens of each sequence attending over its paged 4-bit cache
"""
import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 32  # channels that share a scale and a low value in the 4-bit cache
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _rule(name, op, dtype, B, H, Hkv, Nq, Nk, d, causal, cap=0.0, bias=False, docs=0, pad=0, prefix=0):
    return dict(name=name, op=op, dtype=dtype, B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, causal=causal, cap=cap, bias=bias,
                docs=docs, pad=pad, prefix=prefix)


def _cache(name, op, dtype, B, H, Hkv, Nq, longest, d, page, cap=0.0, bias=False):
    return dict(name=name, op=op, dtype=dtype, B=B, H=H, Hkv=Hkv, Nq=Nq, longest=longest, d=d, page=page, cap=cap, bias=bias)


def listed():
    return [
        # the first chat turn of one user: the smallest prompt, latency counts
        _rule("fwd short capped", "fwd", "fp16", 1, 8, 2, 200, 200, 64, True, cap=30.0),
        # the training shape of the benchmark with a distance bias and a bidirectional prefix
        _rule("fwd bias prefix", "fwd", "fp16", 4, 16, 16, 2048, 2048, 64, True, bias=True, prefix=300),
        # pre-training on packed documents: the long shape of the benchmark, capped, ragged documents, some padding
        _rule("fwd packed docs capped", "fwd", "bf16", 2, 16, 4, 8192, 8192, 128, True, cap=50.0, docs=9, pad=100),
        # wide heads, a prompt chunk behind a cached prefix (more keys than queries), odd lengths
        _rule("fwd wide chunk", "fwd", "bf16", 2, 8, 4, 2001, 3999, 256, True, cap=50.0, bias=True),
        # gradients of the packed pre-training step
        _rule("bwd packed docs", "bwd", "bf16", 2, 16, 4, 8192, 8192, 128, True, docs=9, pad=100),
        # gradients of an encoder with a cap and a distance bias on both sides
        _rule("bwd capped bias", "bwd", "fp16", 4, 16, 16, 2048, 2048, 64, False, cap=30.0, bias=True),
        # a small fine-tuning batch with wide heads, odd length, two documents a row and a prefix
        _rule("bwd wide small", "bwd", "bf16", 2, 4, 2, 777, 777, 256, True, cap=50.0, docs=2, prefix=60),
        # one decoding step of a serving batch: a row for each sequence goes into the cache
        _cache("store step", "store", "bf16", 64, 32, 8, 1, 2000, 128, 64),
        # prompts of a serving batch go into the cache, and the cached rows are read back for the next chunk
        _cache("store prompts", "store", "bf16", 4, 32, 8, 4096, 4096, 128, 64),
        # one token of one short chat: latency counts
        _cache("attend one short", "attend", "fp16", 1, 32, 8, 1, 517, 128, 16, cap=50.0),
        # one decoding step of a busy server: ragged contexts
        _cache("attend batch", "attend", "bf16", 32, 32, 8, 1, 16384, 128, 64),
        # a long document, three speculated tokens, wide heads, a distance bias
        _cache("attend long", "attend", "bf16", 2, 16, 4, 3, 100003, 256, 128, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes spread over the ranges, then halved until it costs no more than the largest listed one."""
    c = _drawn(rng)
    while _cost(c) > 1.0:
        if c["op"] in ("fwd", "bwd"):
            c["docs"], c["pad"], more = c["docs"] if c["docs"] < 4 else 4, c["pad"] // 2, (c["Nk"] - c["Nq"]) // 2
            c["Nq"] = c["Nq"] // 2 + 1
            c["Nk"] = c["Nq"] + more
            c["prefix"] = min(c["prefix"], c["Nk"])
        else:
            c["longest"] = c["longest"] // 2 + 1
            c["Nq"] = min(c["Nq"], c["longest"]) if c["op"] == "store" else c["Nq"]
    return c


def _cost(c):
    """Against the largest listed case of its operator: scores computed densely, or bytes of the cache."""
    if c["op"] in ("fwd", "bwd"):
        return c["B"] * c["H"] * c["Nq"] * c["Nk"] * c["d"] / (2 * 16 * 8192 * 8192 * 128 / 2)
    return work(c)["bytes"] / (1.4e8 if c["op"] == "store" else 3.8e8)


def _drawn(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "store", "attend", "attend"])
    dtype, d = rng.choice(["fp16", "bf16"]), rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 8] if op in ("fwd", "bwd") else [1, 2, 4, 5, 8])
    cap, bias = rng.choice([0.0, 20.0, 50.0]), rng.random() < 0.5
    if op in ("fwd", "bwd"):
        B = rng.randint(1, 4)
        Nq = _log(rng, 1, 6000)
        while B * Hkv * group > 32:
            B, group = max(1, B // 2), group if B > 1 else max(1, group // 2)
        Nk = Nq if rng.random() < 0.6 else min(8000, Nq + _log(rng, 1, 2000))
        docs = rng.randint(1, 12) if Nk == Nq and rng.random() < 0.5 else 0
        return {k: v for k, v in _rule("", op, dtype, B, Hkv * group, Hkv, Nq, Nk, d, rng.random() < 0.7, cap, bias, docs,
                                       rng.randint(0, Nq // 8) if docs else 0,
                                       rng.randint(1, Nk) if rng.random() < 0.3 else 0).items() if k != "name"}
    page = rng.choice([16, 32, 64, 128])
    if op == "store":
        longest = _log(rng, 1, 4096)
        Nq = rng.choice([1, max(1, longest // 3), longest])
        return {k: v for k, v in _cache("", op, dtype, _log(rng, 1, 16), Hkv * group, Hkv, Nq, longest, d, page).items() if k != "name"}
    B = _log(rng, 1, 48)
    return {k: v for k, v in _cache("", op, dtype, B, Hkv * group, Hkv, rng.choice([1, 1, 1, 2, 4, 7]),
                                    _log(rng, 1, max(64, min(60000, 500000 // B))), d, page, cap, bias).items() if k != "name"}


# ------------------------------------------------------------------------------------------ inputs


def _doc_lengths(c):
    """Lengths of the documents of each batch row (they depend on the case alone), and the padding behind them."""
    out = []
    for b in range(c["B"]):
        r = random.Random(1000 * b + c["docs"])
        n = c["Nk"] - c["pad"]
        cuts = sorted(r.randint(0, n) for _ in range(c["docs"] - 1))
        out.append([y - x for x, y in zip([0] + cuts, cuts + [n])])
    return out


def _prefixes(c):
    return [max(1, c["prefix"] - 17 * b) for b in range(c["B"])]


def _lengths(c):
    """Tokens each sequence has in the cache after this step (they depend on the case alone): the first the longest."""
    r = random.Random(c["longest"])
    lo = max(1, c["longest"] // 8)
    return [c["longest"]] + [r.randint(lo, c["longest"]) for _ in range(c["B"] - 1)]


def _starts(c, lens):
    return [max(0, n - c["Nq"]) for n in lens]


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _slopes(c):
    """2^(-8 (h+1) / H): a geometric row of slopes, one a head."""
    h = torch.arange(1, c["H"] + 1, device=DEV, dtype=torch.float32)
    return torch.exp2(-8.0 * h / c["H"]) if c["bias"] else None


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t = TYPES[c["dtype"]]
    s = {"c": c, "scale": 1.0 / math.sqrt(c["d"]), "slopes": _slopes(c)}
    if c["op"] in ("fwd", "bwd"):
        # capped models have larger scores: a wider q
        gain = 3.0 if c["cap"] else 1.0
        s["q"] = (gain * _randn(gen, c["B"], c["H"], c["Nq"], c["d"])).to(t)
        s["k"] = _randn(gen, c["B"], c["Hkv"], c["Nk"], c["d"]).to(t)
        s["v"] = _randn(gen, c["B"], c["Hkv"], c["Nk"], c["d"]).to(t)
        s["ids"] = None
        if c["docs"]:
            rows = [sum(([i] * n for i, n in enumerate(ls)), []) + [-1] * c["pad"] for ls in _doc_lengths(c)]
            s["ids"] = torch.tensor(rows, dtype=torch.int32, device=DEV)
        s["prefix"] = torch.tensor(_prefixes(c), dtype=torch.int32, device=DEV) if c["prefix"] else None
        if c["op"] == "bwd":
            s["dout"] = _randn(gen, c["B"], c["H"], c["Nq"], c["d"]).to(t)
            s["o"], s["lse"] = _plain_fwd(s)
        return s
    lens = _lengths(c)
    per = -(-c["longest"] // c["page"])
    pages = c["B"] * per
    s["table"] = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).view(c["B"], per).contiguous()
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["start"] = torch.tensor(_starts(c, lens), dtype=torch.int32, device=DEV)
    for n in "kv":
        s[n + "_codes"] = torch.randint(0, 256, (pages, c["Hkv"], c["page"], c["d"] // 2), generator=gen, device=DEV, dtype=torch.uint8)
        scale = 0.2 + 0.1 * torch.rand(pages, c["Hkv"], c["page"], c["d"] // GROUP, generator=gen, device=DEV)
        low = -7.5 * scale + 0.3 * _randn(gen, *scale.shape)
        s[n + "_params"] = torch.stack([scale, low], -1).to(t)
    if c["op"] == "store":
        s["k"] = _randn(gen, c["B"], c["Hkv"], c["Nq"], c["d"]).to(t)
        s["v"] = _randn(gen, c["B"], c["Hkv"], c["Nq"], c["d"]).to(t)
        s["count"] = s["lengths"] - s["start"]
        # a step reads back the row that it wrote; prompts read back the whole sequences
        s["from"] = s["start"] if c["Nq"] == 1 else torch.zeros_like(s["start"])
        s["rows"] = 1 if c["Nq"] == 1 else c["longest"]
    else:
        s["q"] = ((3.0 if c["cap"] else 1.0) * _randn(gen, c["B"], c["H"], c["Nq"], c["d"])).to(t)
    return s


# ------------------------------------------------------------------------------------------ plain forms


def _scores(s, q, k):
    """Scores after the cap and the bias in 32 bits (-inf where hidden), and tanh of the capped ones."""
    c = s["c"]
    Nq, Nk = q.shape[2], k.shape[2]
    off = Nk - Nq
    z, th = torch.matmul(q.float(), k.float().transpose(-1, -2)).mul_(s["scale"]), None
    if c["cap"]:
        th = torch.tanh(z.div_(c["cap"]))
        z = th * c["cap"]
    i = torch.arange(Nq, device=q.device)[:, None] + off
    j = torch.arange(Nk, device=q.device)[None, :]
    if s["slopes"] is not None:
        z = z - s["slopes"][None, :, None, None] * (i - j).abs().float()
    see = torch.ones(c["B"], 1, Nq, Nk, dtype=torch.bool, device=q.device)
    if s["ids"] is not None:
        see = see & (s["ids"][:, None, :, None] == s["ids"][:, None, None, :]) & (s["ids"][:, None, None, :] >= 0)
    if c["causal"]:
        near = (j <= i)[None, None]
        if s["prefix"] is not None:
            near = near | (j[None, None] < s["prefix"][:, None, None, None])
        see = see & near
    return z.masked_fill_(~see, -math.inf), th


def _spread(x, H):
    """Each key/value head once for every query head that reads it."""
    return x.repeat_interleave(H // x.shape[1], dim=1)


def _softmax(z):
    m = z.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)  # rows that see nothing
    p = torch.exp(z.sub_(m))
    l = p.sum(-1, keepdim=True)
    return p.div_(torch.where(l > 0, l, torch.ones_like(l))), (m + torch.log(l))[..., 0]


def _plain_fwd(s):
    H = s["c"]["H"]
    z, _ = _scores(s, s["q"], _spread(s["k"], H))
    p, lse = _softmax(z)
    return torch.matmul(p, _spread(s["v"], H).float()).to(s["q"].dtype), lse


def _plain_bwd(s):
    c = s["c"]
    q, k, v = s["q"].float(), _spread(s["k"], c["H"]).float(), _spread(s["v"], c["H"]).float()
    do = s["dout"].float()
    z, th = _scores(s, q, k)
    p = torch.exp(z.sub_(torch.where(torch.isinf(s["lse"]), torch.zeros_like(s["lse"]), s["lse"])[..., None]))
    dv = torch.matmul(p.transpose(-1, -2), do)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * s["o"].float()).sum(-1, keepdim=True)).mul_(p)
    if th is not None:
        ds = ds * (1.0 - th * th)
    dq = torch.matmul(ds, k) * s["scale"]
    dk = torch.matmul(ds.transpose(-1, -2), q) * s["scale"]
    fold = lambda x: x.view(c["B"], c["Hkv"], c["H"] // c["Hkv"], c["Nk"], c["d"]).sum(2)  # noqa: E731
    t = s["q"].dtype
    return dq.to(t), fold(dk).to(t), fold(dv).to(t)


def _held(codes, params, where):
    """The values that cached rows stand for: codes and (scale, low) of the rows at ``where`` (page, row in it)."""
    b, page, row = where
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
    return (None, torch.gather(s["table"].long(), 1, at // c["page"]), at % c["page"]), have


def _coded(x):
    """Codes and (scale, low) of rows x, every step in 32 bits."""
    g = x.float().unflatten(-1, (-1, GROUP))
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale = ((high - low) / 15.0).to(x.dtype).float()
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    inv = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
    q = torch.clamp(torch.round((g - low) * inv), max=15.0).to(torch.uint8).flatten(-2)
    return q[..., 0::2] | (q[..., 1::2] << 4), torch.cat([scale, low], -1).to(x.dtype)


def _plain_store(s):
    c = s["c"]
    (_, page, row), _ = _places(s, s["start"], c["Nq"])
    new = torch.arange(c["Nq"], device=DEV)[None] < s["count"][:, None]
    out = []
    where, have = _places(s, s["from"], s["rows"])
    pick = new.nonzero(as_tuple=True)
    at = (page[pick], row[pick])
    ck, pk = _coded(s["k"])
    cv, pv = _coded(s["v"])
    s["k_codes"][at[0], :, at[1]] = ck.transpose(1, 2)[pick]
    s["k_params"][at[0], :, at[1]] = pk.transpose(1, 2)[pick]
    s["v_codes"][at[0], :, at[1]] = cv.transpose(1, 2)[pick]
    s["v_params"][at[0], :, at[1]] = pv.transpose(1, 2)[pick]
    zero = ~have[:, None, :, None]
    out.append(_held(s["k_codes"], s["k_params"], where).masked_fill(zero, 0.0))
    out.append(_held(s["v_codes"], s["v_params"], where).masked_fill(zero, 0.0))
    return tuple(out)


def _plain_attend(s):
    c = s["c"]
    where, have = _places(s, torch.zeros_like(s["start"]), c["longest"])
    k = _held(s["k_codes"], s["k_params"], where).float()
    v = _held(s["v_codes"], s["v_params"], where).float()
    g = c["H"] // c["Hkv"]
    q = s["q"].float().view(c["B"], c["Hkv"], g, c["Nq"], c["d"])
    z = torch.einsum("bkgid,bkjd->bkgij", q, k) * s["scale"]
    if c["cap"]:
        z = c["cap"] * torch.tanh(z / c["cap"])
    i = (s["lengths"].long()[:, None] - c["Nq"] + torch.arange(c["Nq"], device=DEV)[None])[:, None, None, :, None]
    j = torch.arange(c["longest"], device=DEV)
    if s["slopes"] is not None:
        z = z - s["slopes"].view(1, c["Hkv"], g, 1, 1) * (i - j).abs().float()
    z = z.masked_fill((j > i) | ~have[:, None, None, None, :], -math.inf)
    p, lse = _softmax(z)
    o = torch.einsum("bkgij,bkjd->bkgid", p, v)
    return o.reshape(s["q"].shape).to(s["q"].dtype), lse.reshape(c["B"], c["H"], c["Nq"])


# ------------------------------------------------------------------------------------------ one pass


def run(state):
    s = state
    c = s["c"]
    if own:
        import exact_attention_37_gb300 as fa

        if c["op"] in ("fwd", "bwd"):
            rule = fa.ScoreRule(causal=c["causal"], cap=c["cap"], slopes=s["slopes"], q_doc=s["ids"], k_doc=s["ids"], prefix=s["prefix"])
            if c["op"] == "fwd":
                return fa.forward_rule(s["q"], s["k"], s["v"], rule, scale=s["scale"])
            return fa.backward_rule(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"], rule, scale=s["scale"])
        cache = fa.KV4Cache(s["k_codes"], s["k_params"], s["v_codes"], s["v_params"])
        if c["op"] == "store":
            fa.kv4_append(cache, s["k"], s["v"], s["table"], s["start"], s["count"])
            return fa.kv4_read(cache, s["table"], s["from"], s["rows"], s["lengths"])
        return fa.kv4_attend(s["q"], cache, s["table"], s["lengths"], scale=s["scale"], cap=c["cap"], slopes=s["slopes"])
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "store": _plain_store, "attend": _plain_attend}[c["op"]](s)


def _pairs(c):
    """Visible (query, key) pairs of one head, all batch rows."""
    n = 0
    for b in range(c["B"]):
        pre = _prefixes(c)[b] if c["prefix"] else 0
        runs, at = [], 0
        for length in _doc_lengths(c)[b] if c["docs"] else [c["Nk"]]:
            runs.append((at, at + length))
            at += length
        off = c["Nk"] - c["Nq"]
        for lo, hi in runs:
            first = max(0, lo - off) if c["docs"] else 0
            for i in range(first, min(c["Nq"], hi - off)):
                n += (min(hi, max(i + off + 1, pre)) - lo) if c["causal"] else hi - lo
    return n


def work(case):
    c = case
    if c["op"] in ("fwd", "bwd"):
        q, kv = c["B"] * c["H"] * c["Nq"] * c["d"], c["B"] * c["Hkv"] * c["Nk"] * c["d"]
        rows, ids = c["B"] * c["H"] * c["Nq"], (c["B"] * c["Nk"] if c["docs"] else 0)
        pairs = c["H"] * _pairs(c)
        if c["op"] == "fwd":
            return {"bytes": 2 * (2 * q + 2 * kv) + 4 * (rows + ids), "flops": 4 * c["d"] * pairs}
        return {"bytes": 2 * (4 * q + 4 * kv) + 4 * (rows + ids), "flops": 10 * c["d"] * pairs}
    lens = _lengths(c)
    row = 2 * c["Hkv"] * (c["d"] // 2 + c["d"] // GROUP * 4)  # a cached token: keys and values
    if c["op"] == "store":
        new = sum(n - st for n, st in zip(lens, _starts(c, lens)))
        back = c["B"] if c["Nq"] == 1 else sum(lens)
        out = c["B"] * (1 if c["Nq"] == 1 else c["longest"])
        full = 2 * c["Hkv"] * c["d"] * 2
        return {"bytes": new * (full + row) + back * row + out * full, "flops": 0}
    toks = sum(lens)
    qo = c["B"] * c["H"] * c["Nq"] * (2 * c["d"] * 2 + 4)
    return {"bytes": toks * row + qo, "flops": 4 * c["d"] * c["H"] * c["Nq"] * toks}


# ------------------------------------------------------------------------------------------ in 64 bits


def _exact_rows(s, b, h, q, k, length=None):
    """Scores of one head in 64 bits, its hidden places, and what the cap did to them."""
    c = s["c"]
    u = (q.double() @ k.double().t()) * float(torch.tensor(s["scale"], dtype=torch.float32))
    z = c["cap"] * torch.tanh(u / c["cap"]) if c["cap"] else u
    n, m = u.shape
    pos = torch.arange(m - n if length is None else length - n, m if length is None else length, device=DEV)
    dist = pos[:, None] - torch.arange(m, device=DEV)[None]
    if s["slopes"] is not None:
        z = z - float(s["slopes"][h]) * dist.abs()
    hidden = torch.zeros_like(dist, dtype=torch.bool)
    if c.get("causal", True):
        hidden |= dist < 0
        if c.get("prefix"):
            hidden[:, : int(s["prefix"][b])] = False
    if c.get("docs"):
        kd = s["ids"][b]
        hidden |= (kd[None] != kd[:, None]) | (kd[None] < 0)
    slope = 1.0 - torch.tanh(u / c["cap"]) ** 2 if c["cap"] else None
    return z, hidden, slope


def _exact_held(s, name, b, h, n):
    """Rows 0 .. n - 1 of one cached head of one sequence, in 64 bits; the stored value is rounded to the cache's type."""
    c = s["c"]
    tok = torch.arange(n, device=DEV)
    page = s["table"][b].long()[tok // c["page"]]
    raw = s[name + "_codes"][page, h, tok % c["page"]].long()
    par = s[name + "_params"][page, h, tok % c["page"]].double()
    val = torch.empty(n, c["d"], dtype=torch.float64, device=DEV)
    for ch in range(c["d"]):
        code = (raw[:, ch // 2] >> (4 * (ch % 2))) & 15
        val[:, ch] = par[:, ch // GROUP, 1] + code * par[:, ch // GROUP, 0]
    return val.to(TYPES[c["dtype"]]).double()


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    g = c["H"] // c["Hkv"]
    f8 = dict(dtype=torch.float64, device=DEV)
    if c["op"] == "fwd":
        o, lse = torch.zeros(s["q"].shape, **f8), torch.zeros(s["q"].shape[:3], **f8)
        for b in range(c["B"]):
            for h in range(c["H"]):
                z, hidden, _ = _exact_rows(s, b, h, s["q"][b, h], s["k"][b, h // g])
                z[hidden] = -math.inf
                lse[b, h] = torch.logsumexp(z, -1)
                some = ~torch.isinf(lse[b, h])
                o[b, h, some] = torch.exp(z[some] - lse[b, h, some, None]) @ s["v"][b, h // g].double()
        return o, lse
    if c["op"] == "bwd":
        dq, dk, dv = (torch.zeros(s[n].shape, **f8) for n in "qkv")
        scale = float(torch.tensor(s["scale"], dtype=torch.float32))
        for b in range(c["B"]):
            for h in range(c["H"]):
                z, hidden, slope = _exact_rows(s, b, h, s["q"][b, h], s["k"][b, h // g])
                p = torch.exp(z - s["lse"][b, h].double()[:, None])
                p[hidden] = 0.0
                do = s["dout"][b, h].double()
                dv[b, h // g] += p.t() @ do
                dz = p * (do @ s["v"][b, h // g].double().t() - (do * s["o"][b, h].double()).sum(-1, keepdim=True))
                du = dz * slope * scale if slope is not None else dz * scale
                dq[b, h] = du @ s["k"][b, h // g].double()
                dk[b, h // g] += du.t() @ s["q"][b, h].double()
        return dq, dk, dv
    if c["op"] == "store":
        # the code of a value is chosen in steps of 32 bits by definition; what it stands for is taken in 64
        new = {"k": s["k"], "v": s["v"]}
        outs = []
        for name in "kv":
            x = new[name].float().view(c["B"], c["Hkv"], c["Nq"], -1, GROUP)
            low = x.min(-1, keepdim=True)[0]
            step = ((x.max(-1, keepdim=True)[0] - low) / 15).to(TYPES[c["dtype"]]).float()
            step = step * (step >= 2.0 ** -126)
            code = torch.where(step > 0, torch.round((x - low) * (1 / step)).clamp(max=15), torch.zeros_like(x))
            vals = (low.double() + code.double() * step.double()).to(TYPES[c["dtype"]]).double().flatten(-2)
            out = torch.zeros(c["B"], c["Hkv"], s["rows"], c["d"], **f8)
            for b in range(c["B"]):
                st, n = int(s["start"][b]), int(s["count"][b])
                if c["Nq"] == 1:
                    out[b] = vals[b]
                    continue
                for h in range(c["Hkv"]):
                    out[b, h, :st] = _exact_held(s, name, b, h, st)
                out[b, :, st:st + n] = vals[b, :, :n]
            outs.append(out)
        return tuple(outs)
    o, lse = torch.zeros(s["q"].shape, **f8), torch.zeros(s["q"].shape[:3], **f8)
    for b in range(c["B"]):
        n = int(s["lengths"][b])
        for hk in range(c["Hkv"]):
            k, v = _exact_held(s, "k", b, hk, n), _exact_held(s, "v", b, hk, n)
            for h in range(hk * g, hk * g + g):
                z, hidden, _ = _exact_rows(s, b, h, s["q"][b, h], k, n)
                z[hidden] = -math.inf
                lse[b, h] = torch.logsumexp(z, -1)
                some = ~torch.isinf(lse[b, h])
                o[b, h, some] = torch.exp(z[some] - lse[b, h, some, None]) @ v
    return o, lse
