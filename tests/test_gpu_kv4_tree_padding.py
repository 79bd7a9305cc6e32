"""Rows of a tree call that no tile has: those behind a sequence's count, and all of a sequence without a
token.  They are O = 0 and L = -inf whatever their number, and whatever the outputs held before."""
import pytest
import torch

import exact_attention_37_gb300 as fa

from .drafts import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_attention_37_gb300 import build

    build.build()
    fa.load()


def outputs(B, H, N, d, dtype):
    """Outputs that hold NaN."""
    o = torch.full((B, H, N, d), float("nan"), dtype=dtype, device="cuda")
    lse = torch.full((B, H, N), float("nan"), device="cuda")
    return o, lse


def test_pieces_past_2_31():
    """2^31 pieces of 8 channels, as many as there are 16-byte stores: a counter of 32 bits would see none of them."""
    H, Hkv, N, d, page = 1 << 19, 64, 128, 256, 16
    cache = fa.KV4Cache.empty(1, Hkv, page, d, torch.bfloat16)
    for x in cache.pools:
        x.zero_()
    q = torch.zeros(1, H, N, d, dtype=torch.bfloat16, device="cuda")
    o, lse = outputs(1, H, N, d, torch.bfloat16)
    assert o.numel() // 8 == 1 << 31
    ws = torch.empty(fa.fa_kv4_attend_tree_workspace_size(1, H, Hkv, N, d), dtype=torch.uint8, device="cuda")
    par = i32([[-1] * N])
    fa.fa_kv4_attend_tree(q, cache, i32([[0]]), i32([0]), par, i32([1]), o, lse, ws, d ** -0.5)
    assert all(not bool(o[0, h:h + 4096].any()) for h in range(0, H, 4096))
    assert bool((lse == -float("inf")).all())
    fa.fa_check_device_status()


def call(B, H, Hkv, N, d, lens, count, room, dtype=torch.bfloat16, page=64):
    """A tree call over zeros, and its outputs; room: of the page table, by which the kernel is chosen."""
    pages = [-(-n // page) for n in lens]
    cache = fa.KV4Cache.empty(sum(pages) + 1, Hkv, page, d, dtype)
    for x in cache.pools:
        x.zero_()
    table, at = torch.full((B, -(-room // page)), -1, dtype=torch.int32), 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    table = table.cuda()
    q = torch.zeros(B, H, N, d, dtype=dtype, device="cuda")
    o, lse = outputs(B, H, N, d, dtype)
    ws = torch.empty(fa.fa_kv4_attend_tree_workspace_size(B, H, Hkv, N, d), dtype=torch.uint8, device="cuda")
    args = table, i32(lens), i32([[-1] * N] * B), i32(count)
    return lambda: fa.fa_kv4_attend_tree(q, cache, *args, o, lse, ws, d ** -0.5), o, lse


@pytest.mark.parametrize("B,H,Hkv,N,d", [(1, 16, 2, 128, 256), (3, 8, 2, 40, 128), (33, 32, 2, 20, 128), (160, 32, 1, 10, 64), (70, 4, 1, 9, 256)])
@pytest.mark.parametrize("some", [0, 1, 2])  # sequences with tokens: none, one, most of them
@pytest.mark.parametrize("room", [128, 1 << 18])  # either kernel
def test_every_row_is_written(B, H, Hkv, N, d, some, room):
    """Query heads from fewer than blocks to more than 32 a block; blocks with tiles and without."""
    lens = [(0 if some == 0 or (some == 1 and b != B // 2) else 1 + (37 * b + 90) % 128) for b in range(B)]
    count = [(7 * b + 1) % (N + 1) for b in range(B)]
    run, o, lse = call(B, H, Hkv, N, d, lens, count, room)
    run()
    fa.fa_check_device_status()
    real = torch.zeros(B, N, dtype=torch.bool)
    for b, (n, m) in enumerate(zip(lens, count)):
        for i in range(m if n else 0):
            real[b, i] = n - m + i >= 0
    real = real.cuda()[:, None].expand(B, H, N)
    assert not bool(o.any())
    assert bool((lse[~real] == -float("inf")).all())
    # equal scores: each row sees the prefix and itself
    sees = torch.tensor([max(n - m, 0) + 1 for n, m in zip(lens, count)], device="cuda").view(B, 1, 1).expand(B, H, N)
    assert bool(((lse - sees.log()).abs()[real] <= 1e-4).all())


@pytest.mark.parametrize("H,Hkv,N,d,n", [(64, 8, 128, 256, 1024), (32, 8, 128, 128, 4096)])
def test_padding_costs_no_more_than_rows(H, Hkv, N, d, n):
    """A draft of one token in rows for N takes no longer (by half at most) than one of N."""
    times = []
    for m in (1, N):
        run, _, _ = call(1, H, Hkv, N, d, [n], [m], n)
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(10):
                run()
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        each = []
        for _ in range(6):
            a.record()
            g.replay()
            b.record()
            torch.cuda.synchronize()
            each.append(a.elapsed_time(b))
        times.append(min(each))
    assert times[0] <= 1.5 * times[1], times
