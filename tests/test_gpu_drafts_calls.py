"""How the calls of a server that drafts may be made: in the checked build, from several threads, with
positions and pages of one call in the next on one stream and in a graph that is replayed with new inputs."""
import ctypes
import threading

import pytest
import torch

import exact_attention_37_gb300 as fa
from exact_attention_37_gb300 import _lib

from .drafts import i32
from .test_gpu_kv4_tree import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_attention_37_gb300 import build

    build.build()
    fa.load()


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def state(s):
    return [x.clone() for x in (*s.pages.arrays, *s.cache.pools)]


@pytest.mark.parametrize("room", [900, 1 << 18])  # either kernel for the trees
@pytest.mark.parametrize("d,N,dtype", [(64, 20, torch.bfloat16), (128, 13, torch.float16), (128, 40, torch.bfloat16), (256, 9, torch.bfloat16)])
def test_checked_build_runs_a_step_clean(d, N, dtype, room):
    """Every device-side check silent, and the results those of the release build."""
    from exact_attention_37_gb300 import build

    lib = _lib.open_library(build.build(debug=True))
    s, t = (Step(d=d, N=N, dtype=dtype, room=room, seed=3) for _ in range(2))
    for x in (s, t):
        x.admit()
    want = s.draft()
    B, H, Hkv, N, d, page = t.shape
    par, count, _ = t.t
    p, pages, cache = lambda x: x.data_ptr(), t.pages, t.cache.struct()
    at, st = ctypes.addressof(cache), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    out_count, lens, pos = torch.empty_like(count), torch.empty_like(count), torch.empty(B, N, dtype=torch.int32, device="cuda")
    slots = torch.empty(B, N, dtype=torch.int64, device="cuda")
    m = pages.table.shape[1]
    assert lib.fa_kv4_plan(p(pages.table), p(pages.held), m, p(pages.free), pages.free.shape[0], p(pages.free_count), page, p(t.length),
                           p(count), p(par), p(out_count), p(lens), p(slots), p(pos), B, N, st) == 0
    q, k, o = torch.empty_like(t.q), torch.empty_like(t.k), torch.empty_like(t.q)
    rq, rk = (_lib._rotary_rows(x, y, t.q, t.q.get_device()) for x, y in ((t.q, q), (t.k, k)))
    code = _lib._dtype_code(t.q)
    assert lib.fa_rotary(ctypes.addressof(rq), ctypes.addressof(rk), p(pos), p(t.freqs), 2 * t.freqs.shape[0], 0, 0, 1.0, B, H, Hkv, N, d,
                         code, st) == 0
    assert lib.fa_kv4_append(at, p(k), p(t.v), p(pages.table), m, p(t.length), p(out_count), B, N, st) == 0
    lse = torch.empty(B, H, N, device="cuda")
    ws = torch.empty(lib.fa_kv4_attend_tree_workspace_size(B, H, Hkv, N, d), dtype=torch.uint8, device="cuda")
    assert lib.fa_kv4_attend_tree(p(q), at, p(pages.table), m, p(lens), p(par), p(out_count), p(o), p(lse), 0.0, None, p(ws), ws.numel(), B,
                                  H, N, d ** -0.5, st) == 0
    assert lib.fa_kv4_keep(at, p(pages.table), m, p(t.length), p(t.path), p(t.kept), B, N, st) == 0
    assert lib.fa_check_device_status(st) == 0
    assert same((q, k, o, lse, slots, pos), want) and same(state(t), state(s))
    fa.fa_check_device_status()


def test_steps_from_several_threads():
    """Servers of their own, streams of their own, either kernel for the trees."""
    args = [dict(seed=1, room=900), dict(seed=2, N=40, room=30000), dict(seed=3, d=64, N=17, room=60000), dict(seed=4, d=256, N=9, room=1 << 18)]
    want = []
    for a in args:
        s = Step(**a)
        s.admit()
        want.append([x.clone() for x in s.draft()])
    torch.cuda.synchronize()
    got, err = [None] * 8, []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                s = Step(**args[i % 4])
                s.admit()
                for _ in range(6):  # (again over what was kept: the first step's rows are the draft's)
                    got[i] = s.draft()
            st.synchronize()
        except Exception as e:  # noqa: BLE001
            err.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not err, err
    torch.cuda.synchronize()
    for i in range(8):
        assert same(got[i], want[i % 4])
    fa.fa_check_device_status()


@pytest.mark.parametrize("room", [900, 30000])
def test_a_captured_step_with_new_inputs(room):
    """One graph, replayed for other lengths, trees and rows than it was captured with."""
    N = 21
    live = Step(seed=7, N=N, room=room)
    live.admit()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = live.draft()
    for seed in (8, 9, 10):
        other = Step(seed=seed, N=N, room=room)
        other.admit()
        for x, y in zip((*live.pages.arrays, *live.cache.pools, live.length, live.path, live.kept, live.q, live.k, live.v, *live.t[:2]),
                        (*other.pages.arrays, *other.cache.pools, other.length, other.path, other.kept, other.q, other.k, other.v, *other.t[:2])):
            x.copy_(y)
        g.replay()
        want = other.draft()
        torch.cuda.synchronize()
        assert same(out, want) and same(state(live), state(other))
    fa.fa_check_device_status()


def test_a_server_over_many_steps():
    """Pages come and go over many steps; each step's attention is that of a cache filled at once."""
    s = Step(seed=11, B=9, N=12, room=2000)
    s.admit()
    par, count, _ = s.t
    for step in range(12):
        q, k, o, lse, slots, pos = s.draft()
        s.length.add_(s.kept)
        if step % 4 == 3:  # some requests end and their pages go back; new ones of other lengths come
            s.length[step % 9] = 0
            s.length[(step + 4) % 9].clamp_(max=17)
    table, held = s.pages.table, s.pages.held
    fa.kv4_plan(s.pages, s.shape[5], s.length, i32([0] * 9), 1)
    pages = table[table >= 0].tolist()
    assert len(pages) == len(set(pages)) == int(held.sum())
    free = s.pages.free[: int(s.pages.free_count)].tolist()
    assert sorted(pages + free) == list(range(s.pages.free.shape[0]))
    fa.fa_check_device_status()
