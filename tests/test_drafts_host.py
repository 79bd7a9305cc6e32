"""Rotary positions, page tables and drafted trees without a GPU: angle arithmetic, what the calls
refuse, and pins of the oracle."""
import ctypes
import math
import random

import numpy as np
import pytest
import torch

import exact_attention_37_gb300 as fa
from exact_attention_37_gb300 import _lib
from exact_attention_37_gb300 import build as fabuild
from oracle import drafts, kv4

from .drafts import chain, tree
from .test_kv4_host import BAD_CACHES, cache_struct

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return _lib.load()


# ------------------------------------------------------------------------------------------ rotary


@pytest.mark.parametrize("freq", [1.0, 1e-4, 0.5, 3.2e-7, -0.3, 6.283185307179586, 7.5, 1e6, -2.0 ** -30, 2.0 ** 51 + 0.5])
def test_turns_are_exact_at_every_position(lib, freq):
    t = fa.fa_rotary_turns(freq)
    for pos in (0, 1, -1, 7, 4095, 131072, 10 ** 6 + 3, 2 ** 31 - 1, -2 ** 31):
        got = (t * pos) % 2 ** 64 / 2 ** 64
        off = got - drafts.turns(pos, freq)
        # the fraction is cut to 2^-64 (and, of 1 / (2 pi)'s 128 bits, to |freq| 2^-128) a position
        assert abs(off - round(off)) <= (abs(pos) + 1) * (2.0 ** -64 + abs(freq) * 2.0 ** -127) + 2.0 ** -52


def test_turns_of_tiny_frequencies(lib):
    assert fa.fa_rotary_turns(0.0) == 0 and fa.fa_rotary_turns(-0.0) == 0
    assert fa.fa_rotary_turns(5e-324) == 0 and fa.fa_rotary_turns(1e-25) == 0
    assert fa.fa_rotary_turns(2.0 ** -60) == int(16 / (2 * math.pi))


def rotary_call(lib, **over):
    a = dict(q=256, qo=256, k=512, ko=512, qs=(4096, 1024, 128), qos=(4096, 1024, 128), pos=256, freqs=256, dims=128, amplitude=1.0,
             B=2, H=4, Hkv=4, N=8, d=128, dtype=1, null_q=False, null_k=False)
    a.update(over)
    c3 = ctypes.c_longlong * 3
    q = _lib.RotaryRowsStruct(a["q"], a["qo"], c3(*a["qs"]), c3(*a["qos"]))
    k = _lib.RotaryRowsStruct(a["k"], a["ko"], c3(4096, 1024, 128), c3(4096, 1024, 128))
    return lib.fa_rotary(None if a["null_q"] else ctypes.byref(q), None if a["null_k"] else ctypes.byref(k), vp(a["pos"]), vp(a["freqs"]),
                         a["dims"], 0, 0, a["amplitude"], a["B"], a["H"], a["Hkv"], a["N"], a["d"], a["dtype"], None)


@pytest.mark.parametrize("over,code", [
    (dict(d=96), 2), (dict(dims=8), 2), (dict(dims=24), 2), (dict(dims=144), 2), (dict(dims=0), 2), (dict(dtype=2), 1),
    (dict(B=-1), 1), (dict(N=-1), 1), (dict(H=-1), 1), (dict(Hkv=-1), 1), (dict(amplitude=float("nan")), 1),
    (dict(amplitude=float("inf")), 1), (dict(null_q=True), 1), (dict(null_k=True), 1), (dict(freqs=0), 1), (dict(q=0), 1),
    (dict(ko=0), 1), (dict(q=264), 3), (dict(qo=8), 3), (dict(pos=258), 3), (dict(freqs=260), 3), (dict(qs=(4096, 1024, 132)), 3),
    (dict(qos=(4096, 1020, 128)), 3), (dict(qos=(4096, 0, 128)), 1), (dict(qos=(4096, 1024, 64)), 1), (dict(qs=(-8, 1024, 128)), 1),
    (dict(B=1 << 20, N=1 << 20), 2), (dict(H=65536), 2), (dict(N=0), 0), (dict(B=0), 0), (dict(H=0, Hkv=0), 0)])
def test_rotary_refusals(lib, over, code):
    assert rotary_call(lib, **over) == code


def test_rotary_frequencies():
    f = fa.rotary_freqs(64, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,) and f[0] == 1.0 and f[-1] == 10000.0 ** (-62 / 64)
    assert torch.equal(fa.rotary_freqs(64, scaling="linear", factor=4.0, device="cpu"), f / 4)
    n = fa.rotary_freqs(64, scaling="ntk", factor=4.0, device="cpu")
    assert n[0] == 1.0 and abs(n[-1] / f[-1] - 0.25) < 1e-12
    b = fa.rotary_freqs(64, scaling="bands", factor=8.0, trained=8192, device="cpu")
    turns = 8192 * f / (2 * math.pi)
    assert torch.equal(b[turns >= 4], f[turns >= 4]) and torch.allclose(b[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and bool(((b < f) & (b > f / 8))[mid].all())
    for bad in (dict(dims=8), dict(dims=24), dict(dims=64, scaling="other"), dict(dims=64, base=0.0), dict(dims=64, factor=-1.0),
                dict(dims=64, scaling="bands", low=4.0, high=4.0)):
        with pytest.raises(ValueError):
            fa.rotary_freqs(**bad, device="cpu")


def test_oracle_rotary_keeps_distances():
    """The product of a turned query and key depends on the distance only, and turning back undoes it."""
    rng = np.random.default_rng(0)
    f = fa.rotary_freqs(32, device="cpu").numpy()
    for inter in (False, True):
        q, k = rng.standard_normal((2, 1, 1, 1, 64))
        at = lambda x, p: drafts.rotary(x, np.array([[p]]), f, inter)[0]  # noqa: E731
        assert abs((at(q, 100007) * at(k, 100000)).sum() - (at(q, 7) * at(k, 0)).sum()) < 1e-12
        back = drafts.rotary(at(q, -12345), np.array([[-12345]]), f, inter, backward=True)[0]
        assert np.abs(back - q).max() < 1e-13
        assert np.array_equal(at(q, 9)[..., 32:], q[..., 32:])


# ------------------------------------------------------------------------------------------ the cache's calls


@pytest.mark.parametrize("over,code", BAD_CACHES)
def test_bad_caches_are_refused(lib, over, code):
    c, p = cache_struct(**over), vp(256)
    assert lib.fa_kv4_attend_tree(p, ctypes.byref(c), p, 3, p, p, p, p, p, 0.0, None, p, 1 << 30, 2, 4, 1, 0.1, None) == code
    assert lib.fa_kv4_keep(ctypes.byref(c), p, 3, p, p, p, 2, 5, None) == code


def test_tree_refusals(lib):
    p, z = vp(256), vp(0)
    c = ctypes.byref(cache_struct())

    def at(**o):
        a = {**dict(q=p, c=c, t=p, m=3, l=p, par=p, cnt=p, o=p, s=p, cap=0.0, sl=z, ws=p, b=1 << 30, B=2, H=4, N=1, scale=0.1), **o}
        return lib.fa_kv4_attend_tree(*a.values(), None)

    assert at(H=3) == 1 and at(cap=-1.0) == 1 and at(cap=float("nan")) == 1 and at(scale=0.0) == 1
    assert at(par=z) == 1 and at(q=z) == 1 and at(l=z) == 1 and at(c=None) == 1
    assert at(par=vp(258)) == 3 and at(cnt=vp(257)) == 3 and at(sl=vp(258)) == 3 and at(ws=vp(256 + 16)) == 3
    assert at(ws=z) == 4 and at(b=100) == 4
    assert at(N=129) == 2 and at(B=4097) == 2
    assert at(N=0, par=z) == 0 and at(B=0, par=z) == 0
    assert lib.fa_kv4_attend_tree_workspace_size(2, 4, 2, 128, 64) > 0
    for bad in ((2, 4, 2, 129, 64), (2, 3, 2, 1, 64), (0, 4, 2, 1, 64), (2, 4, 2, 1, 96)):
        assert lib.fa_kv4_attend_tree_workspace_size(*bad) == 0


def test_keep_refusals(lib):
    p, z = vp(256), vp(0)
    c = ctypes.byref(cache_struct())
    assert lib.fa_kv4_keep(None, p, 3, p, p, p, 2, 5, None) == 1
    for args in ((z, p, p), (p, z, p), (p, p, z)):
        assert lib.fa_kv4_keep(c, p, 3, *args, 2, 5, None) == 1
    for args in ((vp(258), p, p), (p, vp(257), p), (p, p, vp(259))):
        assert lib.fa_kv4_keep(c, p, 3, *args, 2, 5, None) == 3
    assert lib.fa_kv4_keep(c, p, 3, p, p, p, 2, 129, None) == 2
    assert lib.fa_kv4_keep(c, p, 3, p, p, p, -1, 5, None) == 1
    assert lib.fa_kv4_keep(c, p, 3, z, z, z, 0, 5, None) == 0 and lib.fa_kv4_keep(c, p, 3, z, z, z, 2, 0, None) == 0


def test_plan_refusals(lib):
    p, z = vp(256), vp(0)

    def at(**o):
        a = {**dict(t=p, h=p, m=3, f=p, nf=9, fc=p, page=16, st=p, ct=p, par=p, oc=p, l=p, sl=p, po=p, B=2, N=5), **o}
        return lib.fa_kv4_plan(*a.values(), None)

    for n in ("t", "h", "f", "fc", "st", "ct", "oc", "l", "sl", "po"):
        assert at(**{n: z}) == 1
    for n in ("t", "h", "f", "fc", "st", "ct", "par", "oc", "l", "po"):
        assert at(**{n: vp(258)}) == 3
    assert at(sl=vp(260)) == 3
    assert at(B=-1) == 1 and at(N=-1) == 1 and at(m=-1) == 1 and at(nf=-1) == 1
    assert at(page=8) == 2 and at(page=48) == 2 and at(page=2048) == 2 and at(B=4097) == 2 and at(N=129) == 2
    assert at(m=1 << 27) == 2 and at(N=1 << 21, B=1 << 11, par=z) == 2
    assert at(B=0) == 0


def test_oracle_chain_is_causal_attention():
    """A draft in which every token follows the one before it is causal attention."""
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((4, 5, 64)), rng.standard_normal((2, 33, 64)), rng.standard_normal((2, 33, 64))
    sl = np.array([0.5, 0.25, 0.1, 0.0])
    for cap in (0.0, 3.0):
        a = drafts.attend_tree(q, k, v, chain(5), 5, 33, 0.2, cap, sl)
        b = kv4.attend(q, k, v, 33, 0.2, True, cap, sl)
        for x, y in zip(a, b):
            assert np.allclose(x, y, rtol=1e-13, atol=1e-13)


def test_oracle_branches_do_not_see_each_other():
    """Each path of a tree is a chain of its own behind the prefix."""
    rng = np.random.default_rng(2)
    par = [-1, 0, 0, 1, 2, -1, 5]
    k, v, q = rng.standard_normal((1, 17, 64)), rng.standard_normal((1, 17, 64)), rng.standard_normal((1, 7, 64))
    o, lse, _, _ = drafts.attend_tree(q, k, v, par, 7, 17, 0.1, slopes=[0.3])
    for path in ([0, 1, 3], [0, 2, 4], [5, 6]):
        at = list(range(10)) + [10 + i for i in path]
        o1, l1, _, _ = drafts.attend_tree(q[:, path], k[:, at], v[:, at], chain(len(path)), len(path), len(at), 0.1, slopes=[0.3])
        assert np.allclose(o[:, path], o1, atol=1e-13) and np.allclose(lse[:, path], l1, atol=1e-13)
    assert drafts.ancestors([-1, -2, 1, 0, 4, 3], 6, 5) == [[0], None, None, [0, 3], None, [0, 3, 5]]
    assert drafts.ancestors([-1, -1, 1], 3, -1) == [None, [1], [1, 2]]


def test_oracle_plan_holds_each_page_once():
    """Pages are in one table or on the stack, never in two places; a growth that is undone leaves the stack as it was."""
    rng = random.Random(3)
    B, room, pages, page = 7, 9, 30, 16
    table, held, free, top = [[-1] * room for _ in range(B)], [0] * B, list(range(pages)), pages
    length = [0] * B
    for _ in range(60):
        count = [rng.choice([0, 1, 1, 20, 40]) for _ in range(B)]
        start = [0 if rng.random() < 0.15 else n for n in length]
        count = [0 if s == 0 and n else c for s, n, c in zip(start, length, count)]
        before = (list(free[:top]), [list(t) for t in table])
        if start == length:
            t2, h2, f2, top2, got, lens, _, _ = drafts.plan(table, held, free, top, page, start, count, 40)
            t3, h3, f3, top3, *_ = drafts.plan(t2, h2, f2, top2, page, start, [0] * B, 40)
            assert (f3[:top3], t3) == before
        table, held, free, top, got, length, slots, _ = drafts.plan(table, held, free, top, page, start, count, 40)
        used = [p for t in table for p in t if p >= 0]
        assert sorted(used + free[:top]) == list(range(pages))
        assert all(h >= -(-n // page) for h, n in zip(held, length))
        assert all((s[i] >= 0) == (i < g) for s, g in zip(slots, got) for i in range(40))


def test_native_calls_refuse_wrong_arguments():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    f = fa.rotary_freqs(64, device="cpu")
    for call in (lambda: fa.rotary(x, x, None, f), lambda: fa.KV4Pages(*[torch.zeros(1, dtype=torch.int32)] * 4),
                 lambda: fa.KV4Pages.empty(2, 3, 4, device="cpu")):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(TypeError):
        fa.rotary(None, None, None, f)
    assert tree(np.random.default_rng(0), 5)[0] == -1
