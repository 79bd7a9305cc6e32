"""A server that drafts, step after step: what each step answers is that of the rows that are cached by then, however
they came there (prompts, accepted branches moved together, pages that went back and came again)."""
import numpy as np
import pytest
import torch

import exact_attention_37_gb300 as fa
from oracle import drafts, kv4

from .drafts import i32, over_bound, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_attention_37_gb300 import build

    build.build()
    fa.load()


class Server:
    """The device's state, and beside it what each sequence has in the cache by the definitions."""

    def __init__(self, d, dtype, room, num_pages, B=7, H=8, Hkv=2, N=12, page=16, seed=0):
        self.rng, self.gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        self.shape, self.dtype = (B, H, Hkv, N, d, page), dtype
        self.pages = fa.KV4Pages.empty(B, -(-room // page), num_pages)
        self.plan = ([[-1] * (-(-room // page)) for _ in range(B)], [0] * B, list(range(num_pages - 1, -1, -1)), num_pages)
        self.cache = fa.KV4Cache.empty(num_pages, Hkv, page, d, dtype)
        for x in self.cache.pools:
            x.zero_()
        self.freqs = fa.rotary_freqs(d)
        self.held = [(np.zeros((Hkv, 0, d)), np.zeros((Hkv, 0, d))) for _ in range(B)]
        self.unserved = 0

    def length(self):
        return [x[0].shape[1] for x in self.held]

    def rows(self, heads, n):
        return torch.randn(self.shape[0], heads, n, self.shape[4], generator=self.gen).to(self.dtype).cuda()

    def stored(self, b, k, v, n):
        return tuple(np.concatenate([old, kv4.values(*kv4.store(x[b, :, :n]), self.dtype)], 1) for old, x in zip(self.held[b], (k, v)))

    def planned(self, count, N, par=None):
        """fa_kv4_plan, against its definition."""
        start = self.length()
        got = fa.kv4_plan(self.pages, self.shape[5], i32(start), i32(count), N, parents=None if par is None else i32(par))
        *self.plan, out, lens, slots, pos = drafts.plan(*self.plan, self.shape[5], start, count, N, par)
        assert [x.tolist() for x in got] == [out, lens, slots, pos]
        self.unserved += sum(m > 0 and o == 0 for m, o in zip(count, out))
        return i32(start), out, *got

    def admit(self, prompts):
        """Prompts of sequences without a token; the others keep what they have."""
        B, _, Hkv, _, _, _ = self.shape
        n = max(prompts)
        start, out, count, _, _, pos = self.planned(prompts, n)
        k, v = self.rows(Hkv, n), self.rows(Hkv, n)
        k = fa.rotary(k, None, pos, self.freqs)[0]
        fa.kv4_append(self.cache, k, v, self.pages.table, start, count)
        for b in range(B):
            self.held[b] = self.stored(b, k, v, out[b])

    def step(self):
        B, H, Hkv, N, d, _ = self.shape
        rng = self.rng
        par = [tree(rng, N) for _ in range(B)]
        count = [int(rng.integers(1, N + 1)) if n else 0 for n in self.length()]
        start, out, count, lens, _, pos = self.planned(count, N, par)
        q, k = fa.rotary(self.rows(H, N), self.rows(Hkv, N), pos, self.freqs)
        v = self.rows(Hkv, N)
        fa.kv4_append(self.cache, k, v, self.pages.table, start, count)
        o, lse = fa.kv4_attend_tree(q, self.cache, self.pages.table, lens, i32(par), count)
        branch = [drafts.ancestors(p, m, n)[int(rng.integers(0, m))] if m else [] for p, m, n in zip(par, out, self.length())]
        fa.kv4_keep(self.cache, self.pages.table, start, i32([x + [0] * (N - len(x)) for x in branch]), i32([len(x) for x in branch]))
        scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
        for b in range(B):
            n, now = self.held[b][0].shape[1], self.stored(b, k, v, out[b])
            ro, rl, a, z = drafts.attend_tree(q[b].double().cpu().numpy(), *now, par[b], out[b], n + out[b], scale)
            go, gl = o[b].double().cpu().numpy(), lse[b].double().cpu().numpy()
            seen = ~np.isinf(rl)
            assert (gl[~seen] == -np.inf).all() and (go[~seen] == 0).all()
            assert over_bound(go, ro, a, z, self.dtype) <= 1
            assert (np.abs(gl[seen] - rl[seen]) <= 3e-5 * np.maximum(1, np.abs(rl[seen]))).all()
            self.held[b] = tuple(x[:, list(range(n)) + [n + i for i in branch[b]]] for x in now)

    def check_cache(self):
        n = max(self.length()) + 3
        got = fa.kv4_read(self.cache, self.pages.table, i32([0] * len(self.held)), n, i32(self.length()))
        for g, which in zip(got, range(2)):
            for b, rows in enumerate(self.held):
                at = rows[which].shape[1]
                assert np.array_equal(g[b, :, :at].double().cpu().numpy(), rows[which]) and not bool(g[b, :, at:].any())


@pytest.mark.parametrize("room,num_pages", [(512, 41), (20000, 48)])  # either kernel for the trees; too few pages for all
@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.float16), (128, torch.bfloat16), (256, torch.bfloat16)])
def test_every_step_answers_for_the_rows_cached_by_then(d, dtype, room, num_pages):
    s = Server(d, dtype, room, num_pages)
    B, H, Hkv, N, _, page = s.shape
    assert fa.fa_kv4_tree_many_rows(B, H, Hkv, N, d, -(-room // page) * page) == (room > 512)
    s.admit([40, 150, 1, 97, 16, 63, 200])
    for i in range(9):
        s.step()
        if i == 2:  # two requests end, one goes back to its first tokens
            s.held[6] = s.held[2] = tuple(x[:, :0] for x in s.held[6])
            s.held[1] = tuple(x[:, :33] for x in s.held[1])
        if i == 4:  # their places are taken by others
            s.admit([0, 0, 170, 0, 0, 0, 250])
        if i == 6:
            s.held[3] = tuple(x[:, :0] for x in s.held[3])
    s.check_cache()
    assert s.unserved > 0  # pages ran out for some
    fa.fa_check_device_status()
