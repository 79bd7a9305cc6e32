"""Trees of drafted tokens over the 4-bit cache, and accepted rows moved together, on the GPU against
their definition (bounds as in the tests of attention over the cache)."""
import numpy as np
import pytest
import torch

import exact_attention_37_gb300 as fa
from oracle import drafts, kv4

from .drafts import chain, i32, over_bound, tree
from .test_gpu_kv4 import filled

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_attention_37_gb300 import build

    build.build()
    fa.load()


def widened(table, room):
    """The table with room for so many tokens: its form then goes by the room."""
    t = torch.full((table.shape[0], room), -1, dtype=torch.int32, device="cuda")
    t[:, : table.shape[1]] = table
    return t


def check(q, cache, table, lens, kv, vv, par, count, **kw):
    scale = float(torch.tensor(q.shape[-1] ** -0.5, dtype=torch.float32))
    o, lse = fa.kv4_attend_tree(q.cuda(), cache, table, i32(lens), i32(par), None if count is None else i32(count), scale=scale, **kw)
    slopes = kw["slopes"].cpu().numpy() if kw.get("slopes") is not None else None
    for b, n in enumerate(lens):
        m = q.shape[2] if count is None else count[b]
        qq = np.nan_to_num(q[b].double().numpy())
        ro, rl, a, z = drafts.attend_tree(qq, kv[b], vv[b], par[b], m, n, scale, kw.get("cap", 0.0), slopes)
        go, gl = o[b].double().cpu().numpy(), lse[b].double().cpu().numpy()
        assert np.isfinite(go).all()
        assert np.array_equal(np.isinf(rl), np.isinf(gl)) and (gl[np.isinf(gl)] < 0).all()
        assert (go[np.isinf(rl)] == 0).all()
        over = over_bound(go, ro, a, z, q.dtype)
        assert over <= 1, f"O of sequence {b}: {over:.3g} of its bound"
        w = ~np.isinf(rl)
        assert (np.abs(gl[w] - rl[w]) <= 3e-5 * np.maximum(1, np.abs(rl[w]))).all()
    fa.fa_check_device_status()
    return o, lse


def queries(B, H, N, d, dtype, seed=1, gain=2.0):
    return (gain * torch.randn(B, H, N, d, generator=torch.Generator().manual_seed(seed))).to(TYPES[dtype])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("H,Hkv,N", [(4, 2, 1), (8, 2, 3), (5, 1, 7), (8, 2, 16), (4, 4, 37), (16, 2, 13), (2, 1, 128), (3, 1, 64)])
@pytest.mark.parametrize("room", [0, 1 << 18])  # either kernel
def test_shapes(d, dtype, H, Hkv, N, room):
    """Ragged lengths and counts: no token, drafts that are all there is, drafts that end behind a page."""
    lens = [0, 1, N, N + 1, 40, 129, 700]
    rng = np.random.default_rng(N)
    count = [min(N, n) if i < 4 else int(rng.integers(1, min(N, n) + 1)) for i, n in enumerate(lens)]
    cache, table, kv, vv, _, _ = filled(H + d + N, dtype, lens, Hkv, 32, d)
    par = [tree(rng, N) for _ in lens]
    check(queries(len(lens), H, N, d, dtype), cache, widened(table, room // 32) if room else table, lens, kv, vv, par, count)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,page,room,H,N", [(64, 16, 1 << 20, 8, 16), (128, 64, 1 << 20, 8, 16), (128, 16, 9000, 4, 21), (256, 128, 1 << 20, 4, 9),
                                             (256, 16, 9000, 8, 32), (128, 1024, 30000, 2, 100), (64, 1024, 30000, 16, 24)])
def test_long_tables(d, page, room, H, N, dtype):
    """Tables with much room, in which the sequences take little or much; drafts across pages and tiles."""
    lens = [0, 5, N, 1000, 3001, 64 + N, 2048 + N // 2]
    rng = np.random.default_rng(d + N)
    count = [min(N, n) for n in lens]
    cache, table, kv, vv, _, _ = filled(d, dtype, lens, 2, page, d)
    par = [tree(rng, N) for _ in lens]
    check(queries(len(lens), H, N, d, dtype), cache, widened(table, -(-room // page)), lens, kv, vv, par, count)


@pytest.mark.parametrize("d,H,N,dtype", [(64, 16, 20, "bf16"), (128, 16, 24, "bf16"), (128, 16, 37, "fp16"), (256, 16, 40, "bf16")])
def test_many_sequences(d, H, N, dtype):
    """More key/value heads than blocks: a block goes through the tiles of several, of one tile and of many."""
    rng = np.random.default_rng(d + N)
    lens = [int(rng.integers(N, 130)) if i % 3 == 0 else int(rng.integers(130, 2600)) for i in range(44)]
    count = [int(rng.integers(1, N + 1)) for _ in lens]
    cache, table, kv, vv, _, _ = filled(N, dtype, lens, 8, 64, d)
    par = [tree(rng, N) for _ in lens]
    q = queries(len(lens), H, N, d, dtype)
    o, lse = check(q, cache, widened(table, 16384 // 64), lens, kv, vv, par, count)
    scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    for _ in range(20):  # blocks meet their waits in another order each time
        again = fa.kv4_attend_tree(q.cuda(), cache, widened(table, 16384 // 64), i32(lens), i32(par), i32(count), scale=scale)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    fa.fa_check_device_status()


def test_a_thousand_short_sequences():
    """Hundreds of key/value heads for each block, many of them without a token; a table without room."""
    d, H, N, B = 64, 4, 17, 1300
    rng = np.random.default_rng(3)
    lens = [0 if i % 5 == 1 else int(rng.integers(1, 90)) for i in range(B)]
    count = [int(rng.integers(0, min(N, n) + 1)) for n in lens]
    cache, table, kv, vv, _, _ = filled(N, "bf16", lens, 1, 16, d)
    par = [tree(rng, N) for _ in lens]
    q = queries(B, H, N, d, "bf16")
    check(q, cache, table, lens, kv, vv, par, count)
    o, lse = fa.kv4_attend_tree(q.cuda(), cache, table[:, :0].contiguous(), i32(lens), i32(par))
    assert not bool(o.any()) and bool((lse == -float("inf")).all())
    fa.fa_check_device_status()


@pytest.mark.parametrize("cap,bias", [(0.0, True), (20.0, False), (1.5, True)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("room,N", [(600, 9), (1 << 20, 40)])
def test_rules(cap, bias, d, room, N):
    H, Hkv, lens = 8, 2, [N, 500, 77, 333]
    cache, table, kv, vv, _, _ = filled(9 + d, "bf16", lens, Hkv, 16, d)
    rng = np.random.default_rng(5)
    slopes = torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H).cuda() if bias else None
    check(queries(4, H, N, d, "bf16", gain=3.0), cache, widened(table, room // 16), lens, kv, vv, [tree(rng, N) for _ in lens],
          [N, N, N // 2, N], cap=cap, slopes=slopes)


def test_negative_and_steep_slopes():
    lens, N, H = [300, 90], 12, 4
    cache, table, kv, vv, _, _ = filled(3, "fp16", lens, 2, 16, 64)
    slopes = torch.tensor([-0.05, 8.0, 0.0, 100.0], device="cuda")
    check(queries(2, H, N, 64, "fp16"), cache, table, lens, kv, vv, [chain(N), tree(np.random.default_rng(1), N)], None, slopes=slopes)


@pytest.mark.parametrize("room", [200, 1 << 20])
@pytest.mark.parametrize("d,N", [(64, 20), (128, 40), (256, 6)])
def test_rows_that_are_no_tokens(room, d, N):
    """Broken parents, rows behind the count, tokens in front of the sequence: nothing seen, nothing shown, NaN queries and all."""
    rng = np.random.default_rng(8)
    lens = [150, 33, 4, 0]
    cache, table, kv, vv, _, _ = filled(4, "bf16", lens, 1, 32, d)
    par = [tree(rng, N) for _ in lens]
    par[0][1], par[0][3], par[0][5] = -2, 3, N + 5       # none, its own parent, a later one
    par[0][2], par[0][4] = 1, 2                          # behind one that is none
    par[1] = [-7] * N
    par[2] = chain(N)                                    # the draft is longer than the sequence
    count = [N, N, N, N]
    q = queries(4, 4, N, d, "bf16")
    none = [drafts.ancestors(p, N, n - N) for p, n in zip(par, lens)]
    for b in range(4):
        for i in range(N):
            if none[b][i] is None:
                q[b, :, i] = float("nan") if i % 2 else float("inf")
    check(q, cache, widened(table, room // 32), lens, kv, vv, par, count)
    assert none[0][:6] == [[0], None, None, None, None, None]
    # counts outside [0, N_q] are clipped
    a = fa.kv4_attend_tree(q.cuda(), cache, table, i32(lens), i32(par), i32([2 ** 31 - 1] * 4))
    b = fa.kv4_attend_tree(q.cuda(), cache, table, i32(lens), i32(par))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    o, lse = fa.kv4_attend_tree(q.cuda(), cache, table, i32(lens), i32(par), i32([-3] * 4))
    assert not bool(o.any()) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("room", [100, 1 << 20])
@pytest.mark.parametrize("d,H,N,dtype", [(64, 2, 6, "bf16"), (128, 8, 20, "bf16"), (256, 4, 12, "fp16"), (128, 4, 7, "fp16")])
def test_values_that_are_not_finite_reach_who_sees_them(room, d, H, N, dtype):
    """A NaN in a drafted key or value: NaN in the rows below it, nothing in its siblings."""
    n = 70
    cache, table, kv, vv, _, _ = filled(6, dtype, [n], 1, 16, d)
    rng = np.random.default_rng(3)
    par = [tree(rng, N)]
    q = queries(1, H, N, d, dtype).cuda()
    args = lambda: (q, cache, widened(table, room // 16), i32([n]), i32(par))  # noqa: E731
    clean_o, clean_l = fa.kv4_attend_tree(*args())
    rows = drafts.ancestors(par[0], N, n - N)
    for which in "kv":
        bad = N // 3
        page, r = int(table[0, (n - N + bad) // 16]), (n - N + bad) % 16
        params = getattr(cache, which + "_params")
        keep = params[page, 0, r].clone()
        params[page, 0, r, 1 if d > 32 else 0, 1] = float("nan")
        o, lse = fa.kv4_attend_tree(*args())
        params[page, 0, r] = keep
        hit = torch.tensor([bad in x for x in rows], device="cuda")
        assert bool(hit.any()) and not bool(hit.all())
        assert torch.equal(o[:, :, ~hit], clean_o[:, :, ~hit]) and torch.equal(lse[:, :, ~hit], clean_l[:, :, ~hit])
        if which == "k":
            assert bool(torch.isnan(o[:, :, hit]).all()) and bool(torch.isnan(lse[:, :, hit]).all())
        else:
            # the NaN is in channels 32 .. 63, and in no other
            nan = torch.isnan(o[:, :, hit])
            assert bool(nan[..., 32:64].all()) and not bool(nan[..., :32].any()) and not bool(nan[..., 64:].any())
            assert torch.equal(o[:, :, hit][~nan], clean_o[:, :, hit][~nan]) and torch.equal(lse, clean_l)


@pytest.mark.parametrize("d,room", [(64, 400), (128, 1 << 20), (256, 1 << 20)])
def test_a_chain_is_attention_of_the_last_tokens(d, room):
    lens, H, N = [300, 17, 250], 8, 5
    cache, table, kv, vv, _, _ = filled(2, "bf16", lens, 2, 16, d)
    q = queries(3, H, N, d, "bf16")
    t = widened(table, room // 16)
    o, lse = check(q, cache, t, lens, kv, vv, [chain(N)] * 3, None)
    o1, l1 = fa.kv4_attend(q.cuda(), cache, t, i32(lens))
    assert torch.allclose(lse, l1, rtol=0, atol=3e-5 * float(l1.abs().max()))
    assert float((o.float() - o1.float()).abs().max()) <= 2.0 ** -6 * float(o1.float().abs().max())


def test_pages_that_are_not_there():
    n, N = 200, 8
    cache, table, kv, vv, _, _ = filled(7, "bf16", [n, n], 1, 16, 64)
    q = queries(2, 2, N, 64, "bf16").cuda()
    table[0, 3] = -1
    o, lse = fa.kv4_attend_tree(q, cache, table, i32([n, n]), i32([chain(N)] * 2))
    with pytest.raises(fa.FaError) as e:
        fa.fa_check_device_status()
    assert e.value.code == 7
    scale = float(torch.tensor(64 ** -0.5, dtype=torch.float32))
    ro, rl, a, z = drafts.attend_tree(q[0].double().cpu().numpy(), kv[0], vv[0], chain(N), N, n, scale, hidden=range(48, 64))
    assert over_bound(o[0].double().cpu().numpy(), ro, a, z, torch.bfloat16) <= 1
    assert np.abs(lse[0].double().cpu().numpy() - rl).max() <= 1e-4


# ------------------------------------------------------------------------------------------ accepted rows


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("page,Hkv,N", [(16, 3, 1), (16, 2, 40), (64, 1, 128), (1024, 2, 9)])
def test_keep_moves_rows_and_nothing_else(d, dtype, page, Hkv, N):
    rng = np.random.default_rng(N + d)
    lens = [N, 2 * N + 5, 300 + N, N + 1]
    cache, table, _, _, _, _ = filled(1, dtype, lens, Hkv, page, d)
    start = [n - N for n in lens]
    kept = [N, int(rng.integers(0, N + 1)), min(3, N), 0]
    path = [[int(x) for x in rng.integers(0, N, N)] for _ in lens]  # any order, the same twice
    path[2][:kept[2]] = sorted(rng.choice(N, kept[2], replace=False).tolist())
    before = [x.clone() for x in cache.pools]
    fa.kv4_keep(cache, table, i32(start), i32(path), i32(kept))
    fa.fa_check_device_status()
    want = [x.clone() for x in before]
    for b in range(4):
        at = lambda t: (int(table[b, t // page]), t % page)  # noqa: E731
        for j in range(kept[b]):
            (p0, r0), (p1, r1) = at(start[b] + path[b][j]), at(start[b] + j)
            for w, x in zip(want, before):
                w[p1, :, r1] = x[p0, :, r0]
    for got, w in zip(cache.pools, want):
        assert torch.equal(got.view(torch.uint8), w.view(torch.uint8))


def test_keep_drops_what_has_no_place():
    cache, table, _, _, _, _ = filled(1, "bf16", [60, 60], 2, 16, 64)
    before = [x.clone() for x in cache.pools]
    fa.kv4_keep(cache, table, i32([40, 40]), i32([[1, -1, 9, 3]] * 2), i32([-5, 99]))
    with pytest.raises(fa.FaError) as e:
        fa.fa_check_device_status()
    assert e.value.code == 7
    # (the second sequence's 99 rows are its 4: rows 0 and 3 have a place to come from)
    p, r = lambda t: int(table[1, t // 16]), lambda t: t % 16  # noqa: E731
    for got, x in zip(cache.pools, before):
        w = x.clone()
        w[p(40), :, r(40)] = x[p(41), :, r(41)]
        assert torch.equal(got.view(torch.uint8), w.view(torch.uint8))
    fa.kv4_keep(cache, table, i32([40, 2 ** 31 - 2]), i32([[0, 1, 2, 3]] * 2), i32([0, 4]))  # behind every table
    with pytest.raises(fa.FaError):
        fa.fa_check_device_status()


def test_refusals():
    cache, table, _, _, _, _ = filled(1, "bf16", [60, 60], 2, 16, 64)
    lens, par, q = i32([60, 60]), i32([[-1, 0]] * 2), queries(2, 4, 2, 64, "bf16").cuda()
    tree_calls = [lambda: fa.kv4_attend_tree(q, cache, table, lens, None), lambda: fa.kv4_attend_tree(q, cache, table, None, par),
                  lambda: fa.kv4_attend_tree(q, cache, table, lens, par[:, :1]), lambda: fa.kv4_attend_tree(q, cache, table, lens, par.long()),
                  lambda: fa.kv4_attend_tree(q, cache, table, lens, par, i32([1])), lambda: fa.kv4_attend_tree(q.half(), cache, table, lens, par),
                  lambda: fa.kv4_attend_tree(q[:, :3], cache, table, lens, par), lambda: fa.kv4_attend_tree(q, cache, table, lens, par.cpu()),
                  lambda: fa.kv4_attend_tree(q, cache, table, lens, par, slopes=torch.ones(3, device="cuda"))]
    keep_calls = [lambda: fa.kv4_keep(cache, table, lens, None, lens), lambda: fa.kv4_keep(cache, table, None, par, lens),
                  lambda: fa.kv4_keep(cache, table, lens, par, None), lambda: fa.kv4_keep(cache, table, lens, par.long(), lens),
                  lambda: fa.kv4_keep(cache, table, lens, par[:1], lens), lambda: fa.kv4_keep(cache, table, lens, par.cpu(), lens)]
    for call in tree_calls + keep_calls:
        with pytest.raises((ValueError, TypeError)):
            call()
    many = torch.zeros(2, 129, dtype=torch.int32, device="cuda")
    for call, code in ((lambda: fa.kv4_attend_tree(q.repeat(1, 1, 65, 1)[:, :, :129].contiguous(), cache, table, lens, many), 2),
                       (lambda: fa.kv4_keep(cache, table, lens, many, lens), 2), (lambda: fa.kv4_attend_tree(q, cache, table, lens, par, cap=-1.0), 1),
                       (lambda: fa.kv4_attend_tree(q, cache, table, lens, par, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), 4)):
        with pytest.raises(fa.FaError) as e:
            call()
        assert e.value.code == code
    o, lse = fa.kv4_attend_tree(q[:, :, :0], cache, table, lens, par[:, :0].contiguous())
    assert o.shape == (2, 4, 0, 64) and lse.shape == (2, 4, 0)
    fa.fa_check_device_status()


# ------------------------------------------------------------------------------------------ together


class Step:
    """What a server that drafts trees does in a step, from pages to the accepted branch."""

    def __init__(self, B=5, H=8, Hkv=2, N=11, d=128, page=16, room=900, dtype=torch.bfloat16, seed=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.shape = (B, H, Hkv, N, d, page)
        self.pages = fa.KV4Pages.empty(B, -(-room // page), B * -(-400 // page))
        self.cache = fa.KV4Cache.empty(self.pages.free.shape[0], Hkv, page, d, dtype)
        for x in self.cache.pools:
            x.zero_()
        self.length = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.freqs = fa.rotary_freqs(d)
        self.prompt = [int(x) for x in rng.integers(1, 200, B)]
        n = max(self.prompt)
        rand = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
        self.pq, self.pk, self.pv = rand(B, H, n, d), rand(B, Hkv, n, d), rand(B, Hkv, n, d)
        self.q, self.k, self.v = rand(B, H, N, d), rand(B, Hkv, N, d), rand(B, Hkv, N, d)
        self.par = [tree(rng, N) for _ in range(B)]
        self.count = [int(x) for x in rng.integers(1, N + 1, B)]
        rows = [drafts.ancestors(p, c, 1000) for p, c in zip(self.par, self.count)]
        self.branch = [r[c - 1] for r, c in zip(rows, self.count)]
        self.path = i32([x + [0] * (N - len(x)) for x in self.branch])
        self.kept = i32([len(x) for x in self.branch])
        self.t = i32(self.par), i32(self.count), i32(self.prompt)

    def admit(self):
        page, (_, _, prompt) = self.shape[5], self.t
        count, lens, _, pos = fa.kv4_plan(self.pages, page, self.length, prompt, self.pk.shape[2])
        _, k = fa.rotary(self.pq, self.pk, pos, self.freqs)
        fa.kv4_append(self.cache, k, self.pv, self.pages.table, self.length, count)
        self.length.copy_(lens)
        return k

    def draft(self, stream=None):
        N, page, (par, count, _) = self.shape[3], self.shape[5], self.t
        count, lens, slots, pos = fa.kv4_plan(self.pages, page, self.length, count, N, parents=par, stream=stream)
        q, k = fa.rotary(self.q, self.k, pos, self.freqs, stream=stream)
        fa.kv4_append(self.cache, k, self.v, self.pages.table, self.length, count, stream=stream)
        o, lse = fa.kv4_attend_tree(q, self.cache, self.pages.table, lens, par, count, stream=stream)
        fa.kv4_keep(self.cache, self.pages.table, self.length, self.path, self.kept, stream=stream)
        return q, k, o, lse, slots, pos


@pytest.mark.parametrize("room", [900, 20000])  # either kernel for the trees
@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16), (256, torch.bfloat16)])
def test_a_step_of_a_server_that_drafts(d, dtype, room):
    s = Step(d=d, dtype=dtype, room=room)
    pk = s.admit()
    q, k, o, lse, slots, pos = s.draft()
    fa.fa_check_device_status()
    N, page = s.shape[3], s.shape[5]
    scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    after = s.length + s.kept
    ck, cv = fa.kv4_read(s.cache, s.pages.table, torch.zeros_like(s.length), 300, after)
    for b in range(s.shape[0]):
        n, c = s.prompt[b], s.count[b]
        hold = lambda x, y: np.concatenate([kv4.values(*kv4.store(t), dtype) for t in (x[b, :, :n], y[b, :, :c])], 1)  # noqa: E731
        kk, vv = hold(pk, k), hold(s.pv, s.v)
        ro, rl, a, z = drafts.attend_tree(q[b].double().cpu().numpy(), kk, vv, s.par[b], c, n + c, scale)
        assert over_bound(o[b].double().cpu().numpy(), ro, a, z, dtype) <= 1
        w = ~np.isinf(rl)
        assert np.abs(lse[b].double().cpu().numpy()[w] - rl[w]).max() <= 1e-4
        rows = drafts.ancestors(s.par[b], c, 0)
        assert pos[b].tolist() == [n + len(r) - 1 if r else -1 for r in rows]
        assert slots[b].tolist() == [fa.fa_kv4_row(s.pages.table[b].tolist(), page, s.cache.num_pages, n + i) if i < c else -1 for i in range(N)]
        # the cache goes on with the accepted branch
        at = list(range(n)) + [n + i for i in s.branch[b]]
        for got, want in ((ck, kk), (cv, vv)):
            assert np.array_equal(got[b, :, :len(at)].double().cpu().numpy(), want[:, at]) and not bool(got[b, :, len(at):].any())


@pytest.mark.parametrize("room", [900, 20000])  # either kernel for the trees
def test_the_step_captured_and_on_a_stream(room):
    s, r = Step(seed=4, room=room), Step(seed=4, room=room)
    want = [x.clone() for x in (s.admit(), *s.draft())]
    r.admit()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = r.draft(st)
    st.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want[1:], got))
    assert all(torch.equal(x, y) for x, y in zip((*s.pages.arrays, *s.cache.pools), (*r.pages.arrays, *r.cache.pools)))
    t = Step(seed=4, room=room)
    t.admit()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = t.draft()
    for _ in range(2):  # (a second replay writes the draft again over the branch that was kept)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want[1:], out))
    assert all(torch.equal(x, y) for x, y in zip((*s.pages.arrays, *s.cache.pools), (*t.pages.arrays, *t.cache.pools)))
    fa.fa_check_device_status()


@pytest.mark.parametrize("room", [900, 20000])  # either kernel for the trees
def test_two_streams_at_once(room):
    """Two servers at the same time, caches and workspaces of their own."""
    a, b = Step(seed=1, N=30, room=room), Step(seed=2, H=4, d=64, dtype=torch.float16)
    c, d = Step(seed=1, N=30, room=room), Step(seed=2, H=4, d=64, dtype=torch.float16)
    for s in (a, b, c, d):
        s.admit()
    want = [a.draft(), b.draft()]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [s.draft(x) for s, x in zip((c, d), st)]
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert all(torch.equal(m, n) for m, n in zip(x, y))


@pytest.mark.parametrize("room", [900, 20000])  # either kernel for the trees
def test_caller_owned_forms(room):
    s = Step(seed=6, room=room)
    s.admit()
    par, count, _ = s.t
    B, H, Hkv, N, d, page = s.shape
    start = s.length
    lens = start + count
    fa.kv4_plan(s.pages, page, start, count, N)
    fa.kv4_append(s.cache, s.k, s.v, s.pages.table, start, count)
    want = fa.kv4_attend_tree(s.q, s.cache, s.pages.table, lens, par, count)
    o, lse = torch.empty_like(s.q), torch.empty(B, H, N, device="cuda")
    ws = torch.empty(fa.fa_kv4_attend_tree_workspace_size(B, H, Hkv, N, d), dtype=torch.uint8, device="cuda")
    fa.fa_kv4_attend_tree(s.q, s.cache, s.pages.table, lens, par, count, o, lse, ws, d ** -0.5)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    pools = [x.clone() for x in s.cache.pools]
    fa.kv4_keep(s.cache, s.pages.table, start, s.path, s.kept)
    moved = [x.clone() for x in s.cache.pools]
    for x, y in zip(s.cache.pools, pools):
        x.copy_(y)
    fa.fa_kv4_keep(s.cache, s.pages.table, start, s.path, s.kept)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(s.cache.pools, moved))


def test_long_sequence_past_2_31_bytes_of_codes():
    """Offsets of a pool of more than 2^32 bytes: the draft lies in its last pages."""
    page, Hkv, d, N = 1024, 8, 256, 5
    pages = 4300
    cache = fa.KV4Cache.empty(pages, Hkv, page, d, torch.bfloat16)
    assert cache.k_codes.numel() > 2 ** 32
    n = 3000
    g = torch.Generator().manual_seed(0)
    table = i32([[pages - 1, 7, pages - 3]])
    k, v = (torch.randn(1, Hkv, n, d, generator=g).to(torch.bfloat16) for _ in range(2))
    fa.kv4_append(cache, k.cuda(), v.cuda(), table, i32([0]))
    kk, vv = (kv4.values(*kv4.store(x[0]), torch.bfloat16) for x in (k, v))
    par = [[-1, 0, 0, 2, -1]]
    q = queries(1, 8, N, d, "bf16")
    check(q, cache, table, [n], [kk], [vv], par, None)
    fa.kv4_keep(cache, table, i32([n - N]), i32([[0, 2, 3, 0, 0]]), i32([3]))
    got, _ = fa.kv4_read(cache, table, i32([n - N]), 3, i32([n]))
    assert np.array_equal(got[0].double().cpu().numpy(), kk[:, [n - 5, n - 3, n - 2]])
