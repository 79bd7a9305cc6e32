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
