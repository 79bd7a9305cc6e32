"""The paged 4-bit cache on the GPU against its definition: what is stored, what is read
back, and attention over it.

Bounds of the attention, as for the other kernels (u = finfo.eps / 2, E = 1e-4 for fp32
sums and exponentials, S half of fp16's smallest step for a P below 2^-14):
u (sum P |v| + |O|) + E sum P |v| + S (sum |v| + 1); the values are exactly what the cache
stands for.  P is relative to a warp's maximum, so at most 1 over a sum of at least 1.
"""
import numpy as np
import pytest
import torch

import exact_attention_37_gb300 as fa
from oracle import kv4

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
S = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_attention_37_gb300 import build

    build.build()
    fa.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(seed, dtype, lens, Hkv, page, d, spare=3):
    """A cache that holds random rows of every sequence, written by the library: (cache,
    page table, values of k and of v for each sequence)."""
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    B, N = len(lens), max(max(lens), 1)
    per = -(-N // page)
    pages = B * per + spare
    table = torch.randperm(pages, generator=g)[: B * per].view(B, per).to(torch.int32)
    cache = fa.KV4Cache.empty(pages, Hkv, page, d, t)
    for x in (cache.k_codes, cache.v_codes):
        x.fill_(255)
    for x in (cache.k_params, cache.v_params):
        x.fill_(float("nan"))  # slots that nothing was written to
    k = (torch.randn(B, Hkv, N, d, generator=g) + torch.randn(1, Hkv, 1, d, generator=g)).to(t)
    v = torch.randn(B, Hkv, N, d, generator=g).to(t)
    fa.kv4_append(cache, k.cuda(), v.cuda(), table.cuda(), i32([0] * B), i32(lens))
    val = [[kv4.values(*kv4.store(x[b, :, :lens[b]]), t) for b in range(B)] for x in (k, v)]
    return cache, table.cuda(), val[0], val[1], k, v


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("page", [16, 128])
def test_append_and_read_are_the_definition(d, dtype, page):
    lens = [1, 37, 300, 0]
    cache, table, kv, vv, _, _ = filled(d, dtype, lens, 3, page, d)
    N = 310
    k, v = fa.kv4_read(cache, table, i32([0] * 4), N, i32(lens))
    fa.fa_check_device_status()
    for b, n in enumerate(lens):
        for got, want in ((k, kv), (v, vv)):
            assert np.array_equal(got[b, :, :n].double().cpu().numpy(), want[b])
            assert bool((got[b, :, n:] == 0).all())
        if n:
            pages = table[b].cpu().numpy()
            assert np.array_equal(kv4.cached(cache, "k", pages, page, n), kv[b])
    # a window inside the sequences
    k2, _ = fa.kv4_read(cache, table, i32([0, 30, 290, 5]), 20, i32(lens))
    assert torch.equal(k2[1, :, :7], k[1, :, 30:37]) and bool((k2[1, :, 7:] == 0).all())
    assert torch.equal(k2[2, :, :10], k[2, :, 290:300])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_special_values(dtype):
    t = TYPES[dtype]
    tiny, huge = (2.0 ** -24, 30000.0) if dtype == "fp16" else (2.0 ** -126, 2.0 ** 125)
    x = torch.zeros(1, 1, 8, 64)
    x[0, 0, 1] = 7.0
    x[0, 0, 2, 5] = tiny
    x[0, 0, 3, ::2], x[0, 0, 3, 1::2] = huge, -huge
    x[0, 0, 4] = torch.linspace(-1, 1, 64)
    x[0, 0, 5] = torch.arange(64) * 0.5      # steps of one: ties
    x[0, 0, 6] = -0.0
    x[0, 0, 7] = 1000 + torch.arange(64) * 2.0 ** -4
    x = x.to(t)
    cache = fa.KV4Cache.empty(1, 1, 16, 64, t)
    fa.kv4_append(cache, x.cuda(), x.cuda(), i32([[0]]), i32([0]))
    k, v = fa.kv4_read(cache, i32([[0]]), i32([0]), 8, i32([8]))
    want = kv4.values(*kv4.store(x[0]), t)
    assert np.array_equal(k[0].double().cpu().numpy(), want) and torch.equal(k, v)


def test_append_leaves_the_rest_as_it_was():
    cache, table, _, _, _, _ = filled(5, "bf16", [40, 70], 2, 16, 64)
    before = [x.clone() for x in (cache.k_codes, cache.k_params, cache.v_codes, cache.v_params)]
    x = torch.randn(2, 2, 9, 64, device="cuda").to(torch.bfloat16)
    fa.kv4_append(cache, x, x, table, i32([40, 10]), i32([3, 0]))
    fa.fa_check_device_status()
    rows = {(int(table[0, p // 16]), p % 16) for p in (40, 41, 42)}
    for a, b in zip(before, (cache.k_codes, cache.k_params, cache.v_codes, cache.v_params)):
        a, b = a.view(torch.uint8).flatten(3).cpu(), b.view(torch.uint8).flatten(3).cpu()
        changed = {(int(p), int(r)) for p, h, r in (a != b).any(-1).nonzero()}
        assert changed == rows


def check_attend(q, cache, table, lens, kv, vv, hidden=None, **kw):
    scale = float(torch.tensor(q.shape[-1] ** -0.5, dtype=torch.float32))
    o, lse = fa.kv4_attend(q.cuda(), cache, table, i32(lens), scale=scale, **kw)
    t = q.dtype
    slopes = kw["slopes"].cpu().numpy() if kw.get("slopes") is not None else None
    for b, n in enumerate(lens):
        ro, rl, a, z = kv4.attend(q[b].double().numpy(), kv[b], vv[b], n, scale, kw.get("causal", True), kw.get("cap", 0.0),
                                  slopes, hidden[b] if hidden else ())
        go, gl = o[b].double().cpu().numpy(), lse[b].double().cpu().numpy()
        assert np.isfinite(go).all()
        assert np.array_equal(np.isinf(rl), np.isinf(gl)) and (gl[np.isinf(gl)] < 0).all()
        over = np.abs(go - ro) / (U[t] * (a + np.abs(ro)) + 1e-4 * a + S[t] * (z + 1))
        assert over.max() <= 1, f"O of sequence {b}: {over.max():.3g} of its bound"
        w = ~np.isinf(rl)
        assert (np.abs(gl[w] - rl[w]) <= 3e-5 * np.maximum(1, np.abs(rl[w]))).all()
    return o, lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("H,Hkv,Nq", [(4, 2, 1), (8, 1, 1), (5, 1, 2), (24, 2, 1), (6, 3, 5), (40, 1, 2), (2, 2, 37)])
def test_attend_shapes(d, dtype, H, Hkv, Nq):
    """Ragged lengths from none on, columns that fill a tile and that do not."""
    lens = [0, 1, 2, 31, 33, 128, 129, 700]
    cache, table, kv, vv, _, _ = filled(H + d + Nq, dtype, lens, Hkv, 32, d)
    g = torch.Generator().manual_seed(H)
    q = (2 * torch.randn(len(lens), H, Nq, d, generator=g)).to(TYPES[dtype])
    check_attend(q, cache, table, lens, kv, vv)
    fa.fa_check_device_status()


@pytest.mark.parametrize("cap,bias,causal", [(0.0, True, True), (20.0, False, True), (1.5, True, False), (0.0, True, False)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_rules(cap, bias, causal, d):
    H, Hkv, Nq, lens = 8, 2, 3, [2, 500, 77]
    cache, table, kv, vv, _, _ = filled(9 + d, "bf16", lens, Hkv, 16, d)
    q = (3 * torch.randn(3, H, Nq, d, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16)
    slopes = torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H).cuda() if bias else None
    check_attend(q, cache, table, lens, kv, vv, cap=cap, slopes=slopes, causal=causal)


@pytest.mark.parametrize("page", [16, 64, 1024])
def test_attend_one_long_sequence_over_many_ctas(page):
    lens = [20011, 3]
    cache, table, kv, vv, _, _ = filled(page, "fp16", lens, 1, page, 128)
    q = torch.randn(2, 4, 1, 128, generator=torch.Generator().manual_seed(1)).to(torch.float16)
    o, lse = check_attend(q, cache, table, lens, kv, vv)
    again = fa.kv4_attend(q.cuda(), cache, table, i32(lens))
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])  # whatever the order of the CTAs


def test_attend_scores_that_rise_and_fall_over_the_tokens():
    """The running maximum moves in every tile, or never again after the first."""
    n, d = 3000, 64
    for sign in (1.0, -1.0):
        ramp = sign * torch.linspace(-1, 1, n)[None, None, :, None]
        u = torch.ones(d) / d ** 0.5
        k = (30 * ramp * u).to(torch.float16)
        v = torch.randn(1, 1, n, d, generator=torch.Generator().manual_seed(2)).to(torch.float16)
        cache = fa.KV4Cache.empty(n // 16 + 1, 1, 16, d, torch.float16)
        table = torch.arange(n // 16 + 1, dtype=torch.int32, device="cuda")[None]
        fa.kv4_append(cache, k.cuda(), v.cuda(), table, i32([0]))
        kv, vv = ([kv4.values(*kv4.store(x[0]), torch.float16)] for x in (k, v))
        q = (40 * u).expand(1, 2, 1, d).to(torch.float16).contiguous()
        check_attend(q, cache, table, [n], kv, vv)


def test_a_bias_at_positions_that_fp32_does_not_hold():
    """Distances are those of the integers: 2^24 tokens of the sequence repeat the same pages,
    and what a steep bias leaves are the last ones."""
    page, d, n = 1024, 64, 2 ** 24 + 3 * 1024 + 517
    cache, table, kv, vv, _, _ = filled(21, "fp16", [4096], 1, page, d)
    many = -(-n // page)
    pages = table[0, torch.arange(many, device="cuda") % 4][None].contiguous()
    q = torch.randn(1, 2, 3, d, generator=torch.Generator().manual_seed(1)).to(torch.float16)
    slopes = torch.tensor([0.25, 1.0], device="cuda")
    scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    o, lse = fa.kv4_attend(q.cuda(), cache, pages, i32([n]), scale=scale, slopes=slopes)
    fa.fa_check_device_status()
    # the last 2048 tokens alone: a bias of 512 hides the others
    at = np.arange(n - 2048, n) % 4096
    ro, rl, a, z = kv4.attend(q[0].double().numpy(), kv[0][:, at], vv[0][:, at], 2048, scale, True, 0.0, [0.25, 1.0])
    go, gl = o[0].double().cpu().numpy(), lse[0].double().cpu().numpy()
    assert (np.abs(go - ro) <= U[q.dtype] * (a + np.abs(ro)) + 1e-4 * a + S[q.dtype] * (z + 1)).all()
    assert (np.abs(gl - rl) <= 3e-5 * np.maximum(1, np.abs(rl))).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("k_size,v_size", [(1.0, 2.0 ** 16), (2.0 ** 13, 1.0), (2.0 ** 26, 2.0 ** 26), (2.0 ** -60, 2.0 ** -60)])
def test_attend_values_far_from_one(d, k_size, v_size):
    """bf16 values near the ends of the range, large ones in some tokens only."""
    t, n, page = torch.bfloat16, 700, 16
    g = torch.Generator().manual_seed(d)
    k, v = (torch.randn(1, 2, n, d, generator=g) for _ in range(2))
    for x, size in ((k, k_size), (v, v_size)):
        if size > 1:
            x[:, :, ::7] *= size
        else:
            x *= size
    k, v = k.to(t), v.to(t)
    cache = fa.KV4Cache.empty(64, 2, page, d, t)
    table = torch.randperm(64, generator=g)[None].to(torch.int32).cuda()
    fa.kv4_append(cache, k.cuda(), v.cuda(), table, i32([0]))
    kv, vv = ([kv4.values(*kv4.store(x[0]), t)] for x in (k, v))
    q = (torch.randn(1, 4, 2, d, generator=g) / k_size).to(t)
    check_attend(q, cache, table, [n], kv, vv)


def test_lengths_outside_the_table_are_clipped():
    cache, table, kv, vv, _, _ = filled(3, "bf16", [64, 64], 1, 16, 64)
    q = torch.randn(2, 1, 1, 64, device="cuda").to(torch.bfloat16)
    a = fa.kv4_attend(q, cache, table, i32([64, 0]))
    b = fa.kv4_attend(q, cache, table, i32([2 ** 31 - 1, -7]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tokens_without_a_page_are_dropped_hidden_and_recorded():
    lens = [100, 60]
    cache, table, kv, vv, k, v = filled(11, "bf16", lens, 2, 16, 64)
    pages = cache.num_pages
    bad = table.clone()
    bad[0, 2], bad[0, 6], bad[1, 0] = pages, -1, 2 ** 31 - 1
    gone = [list(range(32, 48)) + list(range(96, 100)), list(range(16))]
    q = torch.randn(2, 4, 1, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)

    def recorded():
        with pytest.raises(fa.FaError) as e:
            fa.fa_check_device_status()
        assert e.value.code == 7 and e.value.detail[0] == 64 and e.value.detail[1] == 0x108
        fa.fa_check_device_status()  # cleared

    check_attend(q, cache, bad, lens, kv, vv, hidden=gone)
    recorded()
    a, b = fa.kv4_read(cache, bad, i32([0, 0]), 100, i32(lens))
    recorded()
    a0, _ = fa.kv4_read(cache, table, i32([0, 0]), 100, i32(lens))
    for n in range(2):
        keep = [p for p in range(lens[n]) if p not in gone[n]]
        assert torch.equal(a[n, :, keep], a0[n, :, keep]) and bool((a[n, :, gone[n]] == 0).all())
    before = [x.clone() for x in (cache.k_codes, cache.v_codes)]
    fa.kv4_append(cache, k[:, :, :16].cuda(), v[:, :, :16].cuda(), bad, i32([32, 0]))
    recorded()
    assert torch.equal(before[0], cache.k_codes) and torch.equal(before[1], cache.v_codes)
    fa.kv4_append(cache, k[:, :, :4].cuda(), v[:, :, :4].cuda(), table, i32([-4, 16 * table.shape[1]]))
    recorded()
    assert torch.equal(before[0], cache.k_codes) and torch.equal(before[1], cache.v_codes)


def test_a_run_of_them_together():
    """A prompt, then steps of one token: what attends is what was stored, with the rule of
    the prompt's forward pass."""
    t, B, H, Hkv, d, page = torch.bfloat16, 2, 4, 2, 128, 16
    g = torch.Generator().manual_seed(4)
    lens, steps = [45, 16], 5
    N = max(lens) + steps
    k, v = (torch.randn(B, Hkv, N, d, generator=g).to(t) for _ in range(2))
    q = torch.randn(B, H, N, d, generator=g).to(t)
    per = -(-N // page)
    table = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32).cuda()
    cache = fa.KV4Cache.empty(B * per, Hkv, page, d, t)
    slopes = torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H).cuda()
    fa.kv4_append(cache, k.cuda(), v.cuda(), table, i32([0, 0]), i32(lens))
    # the prompt over the cached values equals the plain rule on them
    kk, vv = fa.kv4_read(cache, table, i32([0, 0]), lens[0], i32(lens))
    po, pl = fa.forward_rule(q[:1, :, :lens[0]].contiguous().cuda(), kk[:1], vv[:1], fa.ScoreRule(causal=True, cap=9.0, slopes=slopes))
    ao, al = fa.kv4_attend(q[:1, :, :lens[0]].contiguous().cuda(), cache, table[:1].contiguous(), i32(lens[:1]), cap=9.0, slopes=slopes)
    # two kernels with their own roundings of P and O: each within u (sum P |v| + |O|) <= 2 u max |v|
    assert float((po.float() - ao.float()).abs().max()) <= 4 * 2.0 ** -8 * float(vv.float().abs().max())
    assert float((pl - al).abs().max()) <= 6e-5 * max(1.0, float(pl.abs().max()))
    for s in range(steps):
        now = [n + s for n in lens]
        at = lambda x: torch.stack([x[b, :, now[b]:now[b] + 1] for b in range(B)]).contiguous()  # noqa: E731
        fa.kv4_append(cache, at(k).cuda(), at(v).cuda(), table, i32(now))
        have = [n + 1 for n in now]
        kv, vv = ([kv4.values(*kv4.store(x[b, :, :have[b]]), t) for b in range(B)] for x in (k, v))
        check_attend(at(q), cache, table, have, kv, vv, cap=9.0, slopes=slopes)
    fa.fa_check_device_status()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rows_at_addresses_of_16_bytes_only(d, dtype):
    """The accesses of 32 bytes are left out where k, v or the outputs do not allow them."""
    t, page, n = TYPES[dtype], 32, 75
    g = torch.Generator(device="cuda").manual_seed(d)
    rows = 2 * 3 * n * d

    def at(offset):
        x = torch.empty(rows + 16, dtype=t, device="cuda")[offset:offset + rows].view(2, 3, n, d)
        assert x.data_ptr() % 32 == 2 * offset
        return x

    k, v = torch.randn(2, 3, n, d, generator=g, device="cuda").to(t), torch.randn(2, 3, n, d, generator=g, device="cuda").to(t)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    start, lens = i32([0, 0]), i32([n, n - 9])
    out = []
    for offset in (0, 8):
        cache = fa.KV4Cache.empty(6, 3, page, d, t)
        for x in cache.pools:
            x.zero_()
        kk, vv = at(offset), at(offset)
        kk.copy_(k), vv.copy_(v)
        fa.kv4_append(cache, kk, vv, table, start)
        ko, vo = at(offset), at(8 - offset)
        fa.fa_kv4_read(cache, table, start, lens, ko, vo)
        out.append([*(x.clone() for x in cache.pools), ko.clone(), vo.clone()])
    fa.fa_check_device_status()
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d,H,Hkv,Nq", [(64, 4, 2, 1), (64, 16, 2, 3), (64, 32, 1, 1), (128, 4, 4, 1), (128, 12, 1, 1), (256, 4, 2, 2),
                                        (256, 9, 1, 1)])
@pytest.mark.parametrize("longest", [1, 100, 129, 250, 500, 1000, 1030, 2040, 4096])
def test_clusters_of_every_size_and_what_lies_beyond(d, H, Hkv, Nq, longest):
    """Few and many pieces a sequence, some of a cluster's CTAs with none, sequences without a
    token among them, a bias and a cap."""
    t, lens = torch.bfloat16, [longest, 0, max(1, longest // 3)]
    cache, table, kv, vv, _, _ = filled(d + longest, "bf16", lens, Hkv, 64, d)
    q = (2 * torch.randn(3, H, Nq, d, generator=torch.Generator().manual_seed(longest))).to(t)
    slopes = torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H).cuda()
    o, lse = check_attend(q, cache, table, lens, kv, vv, cap=8.0, slopes=slopes)
    again = fa.kv4_attend(q.cuda(), cache, table, i32(lens), scale=float(torch.tensor(d ** -0.5, dtype=torch.float32)), cap=8.0, slopes=slopes)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    fa.fa_check_device_status()


@pytest.mark.parametrize("B,H,Hkv,Nq,longest,d", [(300, 3, 3, 1, 700, 128), (37, 4, 2, 5, 3000, 64), (5, 4, 1, 9, 6000, 128),
                                                   (40, 6, 3, 1, 1500, 256), (3, 2, 2, 1, 20000, 64)])
def test_stretches_that_cut_units_anywhere(B, H, Hkv, Nq, longest, d):
    """More units than CTAs, as many, and fewer: a CTA's stretch cuts its first unit, its last,
    both, or holds a part of one; sequences without a token among them."""
    g = torch.Generator().manual_seed(longest)
    lens = [longest] + torch.randint(0, longest, (B - 1,), generator=g).tolist()
    lens[1 + B // 2] = 0
    cache, table, kv, vv, _, _ = filled(d, "bf16", lens, Hkv, 64, d)
    q = (2 * torch.randn(B, H, Nq, d, generator=g)).to(torch.bfloat16)
    o, lse = check_attend(q, cache, table, lens, kv, vv)
    ws = torch.full((fa.fa_kv4_attend_workspace_size(B, H, Hkv, Nq, d),), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere
    again = fa.kv4_attend(q.cuda(), cache, table, i32(lens), scale=float(torch.tensor(d ** -0.5, dtype=torch.float32)), workspace=ws)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    fa.fa_check_device_status()
