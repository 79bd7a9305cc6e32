"""Keys and values that are not finite under a tree of drafted tokens: in the draft they reach the rows below them, in
the prefix all rows of the tree, and nothing else, with either kernel."""
import numpy as np
import pytest
import torch

import exact_attention_37_gb300 as fa
from oracle import drafts

from .drafts import i32, tree
from .test_gpu_kv4 import filled
from .test_gpu_kv4_tree import TYPES, widened

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_attention_37_gb300 import build

    build.build()
    fa.load()


# (heads of two key/value heads, drafted tokens, room, whether the kernel for many rows takes it): its rows one, two and four times over
CASES = [(64, 8, 20, 1 << 20, True), (64, 16, 6, 1 << 20, True), (64, 32, 6, 1 << 20, True), (64, 8, 20, 512, False),
         (128, 8, 6, 1 << 20, True), (128, 16, 6, 1 << 20, True), (128, 16, 13, 1 << 20, True), (128, 8, 9, 512, False),
         (256, 8, 6, 1 << 20, True), (256, 16, 10, 1 << 20, True), (256, 8, 9, 512, False)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,H,N,room,many", CASES)
def test_who_sees_them(d, H, N, room, many, dtype):
    lens, page = [70, 150, 41], 16
    B, Hkv = len(lens), 2
    assert fa.fa_kv4_tree_many_rows(B, H, Hkv, N, d, room) == many
    cache, table, *_ = filled(d + N, dtype, lens, Hkv, page, d)
    t = widened(table, room // page)
    rng = np.random.default_rng(N)
    par, count = [tree(rng, N) for _ in lens], [N - 1, N, N - 2]
    par[0][2] = -5  # no token of the tree, nor what hangs below it
    q = (2 * torch.randn(B, H, N, d, generator=torch.Generator().manual_seed(1))).to(TYPES[dtype]).cuda()
    call = lambda: fa.kv4_attend_tree(q, cache, t, i32(lens), i32(par), i32(count))  # noqa: E731
    clean_o, clean_l = call()
    rows = drafts.ancestors(par[0], count[0], lens[0] - count[0])
    head, other = slice(0, H // Hkv), slice(H // Hkv, H)  # the first key/value head's, in the first sequence
    for tok, value in [(11, "nan"), (0, "inf"), (37, "-inf"), (lens[0] - count[0] + 1, "nan"), (lens[0] - count[0] + 1, "inf")]:
        drafted = tok - (lens[0] - count[0])
        hit = torch.tensor([x is not None and (drafted < 0 or drafted in x) for x in rows], device="cuda")
        assert bool(hit.any()) and not bool(hit.all())
        for which in "kv":
            params, at = getattr(cache, which + "_params"), (int(table[0, tok // page]), 0, tok % page)
            keep = params[at].clone()
            params[at][1, 0], params[at][1, 1] = 0, float(value)  # channels 32 .. 63
            o, lse = call()
            params[at] = keep
            # other sequences, other heads, other rows
            assert torch.equal(o[1:], clean_o[1:]) and torch.equal(lse[1:], clean_l[1:])
            assert torch.equal(o[0, other], clean_o[0, other]) and torch.equal(lse[0, other], clean_l[0, other])
            assert torch.equal(o[0, head][:, ~hit], clean_o[0, head][:, ~hit]) and torch.equal(lse[0, head][:, ~hit], clean_l[0, head][:, ~hit])
            got = o[0, head][:, hit]
            if which == "v":
                assert not bool(torch.isfinite(got[..., 32:64]).any())
                if value == "nan" or drafted >= 0:
                    assert bool(torch.isnan(got[..., 32:64]).all())
                else:
                    assert not bool((got[..., 32:64] == -float(value)).any())
                assert torch.equal(got[..., :32], clean_o[0, head][:, hit][..., :32])
                assert torch.equal(got[..., 64:], clean_o[0, head][:, hit][..., 64:])
                assert torch.equal(lse, clean_l)
            elif value == "nan":
                assert bool(torch.isnan(got).all()) and bool(torch.isnan(lse[0, head][:, hit]).all())
    fa.fa_check_device_status()
