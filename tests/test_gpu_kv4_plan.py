"""Page tables made on the GPU against their definition in plain Python."""
import random

import numpy as np
import pytest
import torch

import exact_attention_37_gb300 as fa
from oracle import drafts

from .drafts import i32, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_attention_37_gb300 import build

    build.build()
    fa.load()


def check(state, page, start, count, N, parents=None):
    """The call against the oracle; returns the new state as lists."""
    table, held, free, top = state
    want = drafts.plan(table, held, free, top, page, start, count, N, parents)
    room = len(table[0])
    pages = fa.KV4Pages(i32(table).view(len(table), room), i32(held), i32(free), i32([top]))
    got = fa.kv4_plan(pages, page, i32(start), i32(count), N, None if parents is None else i32(parents).view(len(table), N))
    assert [x.dtype for x in got] == [torch.int32, torch.int32, torch.int64, torch.int32]
    names = ("table", "held", "free", "free_count", "count", "lengths", "slots", "positions")
    have = (pages.table, pages.held, pages.free, pages.free_count, *got)
    for n, x, w in zip(names, have, want):
        w = np.array([w] if n == "free_count" else w, dtype=np.int64).reshape(tuple(x.shape))
        assert np.array_equal(x.cpu().numpy().astype(np.int64), w), n
    return want[:4], got


@pytest.mark.parametrize("B,room,pages,page,N", [(1, 1, 1, 16, 1), (3, 5, 9, 16, 40), (7, 9, 30, 64, 300), (70, 40, 900, 16, 33),
                                                 (600, 6, 1500, 32, 5), (33, 70, 1500, 16, 600), (4096, 3, 8000, 16, 4)])
def test_steps_of_a_server(B, room, pages, page, N):
    """Sequences grow, end and start again; pages run out and come back."""
    rng = random.Random(B)
    state = ([[-1] * room for _ in range(B)], [0] * B, rng.sample(range(pages), pages), pages)
    length = [0] * B
    for step in range(6):
        end = [rng.random() < 0.2 for _ in range(B)]
        start = [0 if e else n for e, n in zip(end, length)]
        count = [0 if e else rng.choice([0, 1, rng.randint(0, N)]) for e in end]
        state, got = check(state, page, start, count, N)
        length = got[1].tolist()


@pytest.mark.parametrize("B,N", [(1, 1), (5, 7), (40, 24), (3, 128), (300, 64)])
def test_trees(B, N):
    rng = np.random.default_rng(B)
    par = [tree(rng, N) for _ in range(B)]
    par[0][N // 2] = -2            # no token, nor what follows it
    par[-1][-1] = N - 1            # its own parent
    count = [int(rng.integers(0, N + 1)) for _ in range(B)]
    count[0] = N
    start = [int(rng.integers(0, 200)) for _ in range(B)]
    room = -(-(200 + N) // 16)
    pages = B * room
    held = [-(-s // 16) for s in start]
    order = list(rng.permutation(pages))
    table = [[int(order.pop()) if p < h else -1 for p in range(room)] for h in held]
    free = [int(x) for x in order] + [0] * (pages - len(order))
    check((table, held, free, len(order)), 16, start, count, N, par)


def test_too_few_pages_and_too_short_tables():
    # the second needs more than its table has; the third takes the last two; the fourth wants one; the fifth none
    table = [[0, -1, -1], [1, -1, -1], [2, -1, -1], [3, -1, -1], [4, -1, -1]]
    state = (table, [1] * 5, [9, 8, 7, 7, 7], 2)
    got = check(state, 16, [16, 16, 10, 16, 3], [0, 40, 38, 1, 5], 40)[1]
    assert got[0].tolist() == [0, 0, 38, 0, 5]
    # the first that does not fit holds up the smaller one behind it
    got = check(state, 16, [16, 16, 16, 16, 3], [1, 32, 1, 0, 5], 40)[1]
    assert got[0].tolist() == [1, 0, 0, 0, 5]
    # pages that one sequence gives back serve another in the same call
    got = check(([[5, 6, 4], [-1] * 3], [3, 0], [0, 0, 0], 0), 16, [0, 0], [0, 48], 48)[1]
    assert got[0].tolist() == [0, 48]


def test_odd_values_stay_inside():
    """Values that no server would have: clipped, and nothing outside the arrays is touched."""
    state = ([[3, 4], [5, 6]], [7, -2], [1, 2, 0, 0], 9)
    pages = [i32(state[0]).view(2, 2), i32(state[1]), i32(state[2]), i32([state[3]])]
    room = [torch.full((x.numel() + 64,), 77, dtype=torch.int32, device="cuda") for x in pages]
    for r, x in zip(room, pages):
        r[32:32 + x.numel()] = x.flatten()
    view = [r[32:32 + x.numel()].view(x.shape) for r, x in zip(room, pages)]
    fa.kv4_plan(fa.KV4Pages(*view), 16, i32([2 ** 31 - 1, -5]), i32([2 ** 31 - 1, -3]), 3)
    # more pages on the stack than it has room for: the last ones are dropped
    fa.kv4_plan(fa.KV4Pages(*view), 16, i32([0, 0]), i32([0, 3]), 3)
    torch.cuda.synchronize()
    for r, x in zip(room, pages):
        assert bool((r[:32] == 77).all()) and bool((r[32 + x.numel():] == 77).all())


def test_empty_sizes_and_refusals():
    p = fa.KV4Pages.empty(0, 4, 8)
    out = fa.kv4_plan(p, 16, i32([]), i32([]), 5)
    assert out[2].shape == (0, 5)
    p = fa.KV4Pages.empty(2, 4, 8)
    out = fa.kv4_plan(p, 16, i32([16, 0]), i32([5, 5]), 0)  # N = 0: counts are clipped to none
    assert out[0].tolist() == [0, 0] and p.held.tolist() == [1, 0] and out[2].shape == (2, 0)
    p = fa.KV4Pages.empty(2, 0, 8)
    assert fa.kv4_plan(p, 16, i32([0, 0]), i32([1, 0]), 1)[0].tolist() == [0, 0]
    p = fa.KV4Pages.empty(2, 4, 8)
    ok = i32([0, 0])
    for call in (lambda: fa.kv4_plan(p, 16, None, ok, 1), lambda: fa.kv4_plan(p, 16, ok, ok.long(), 1), lambda: fa.kv4_plan(p, 16, ok, i32([0]), 1),
                 lambda: fa.kv4_plan(p, 16, ok, ok, -1), lambda: fa.kv4_plan(p, 16, ok, ok, 3, parents=i32([[0], [0]])),
                 lambda: fa.KV4Pages(p.table, p.held, p.free.long(), p.free_count), lambda: fa.KV4Pages(p.table, p.held[:1], p.free, p.free_count),
                 lambda: fa.KV4Pages(p.table.cpu(), p.held, p.free, p.free_count), lambda: fa.KV4Pages(p.table[:, ::2], p.held, p.free, p.free_count)):
        with pytest.raises((ValueError, TypeError)):
            call()
    for call in (lambda: fa.kv4_plan(p, 24, ok, ok, 1), lambda: fa.kv4_plan(p, 16, ok, ok, 129, parents=torch.zeros(2, 129, dtype=torch.int32, device="cuda"))):
        with pytest.raises(fa.FaError) as e:
            call()
        assert e.value.code == 2


def test_caller_owned_form_streams_and_capture():
    B, N, page = 20, 900, 16
    start, count = i32([7 * b for b in range(B)]), i32([45 * b for b in range(B)])
    make = lambda: fa.KV4Pages.empty(B, 80, 1200)  # noqa: E731
    p = make()
    want = fa.kv4_plan(p, page, start, count, N)
    r = make()
    out = [torch.empty_like(x) for x in want]
    fa.fa_kv4_plan(r, page, start, count, None, *out)
    s = torch.cuda.Stream()
    t = make()
    s.wait_stream(torch.cuda.current_stream())
    other = fa.kv4_plan(t, page, start, count, N, stream=s)
    s.synchronize()
    for a, b in ((out, r), (other, t)):
        assert all(torch.equal(x, y) for x, y in zip((*a, *b.arrays), (*want, *p.arrays)))
    # captured: the pages are changed in place, replay after replay
    c, st, ct = make(), torch.zeros_like(start), torch.full_like(count, 30)
    g = torch.cuda.CUDAGraph()
    warm = [x.clone() for x in c.arrays]
    with torch.cuda.graph(g):
        _, lens, _, _ = fa.kv4_plan(c, page, st, ct, N)
        st.copy_(lens)
    assert all(torch.equal(x, y) for x, y in zip(warm, c.arrays))
    for n in range(3):
        g.replay()
        assert st.tolist() == [30 * (n + 1)] * B and c.held.tolist() == [-(-30 * (n + 1) // page)] * B
    assert int(c.free_count) == 1200 - B * 6 and len(set(c.table[:, :6].flatten().tolist())) == 6 * B
