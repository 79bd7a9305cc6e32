"""NaN in what a row sees comes out of the calls with a score rule and of the cache's: O, L and
the gradients say so, as the plain calls' O and gradients do, whatever the cap and its form of
the tanh, and the rows that do not see it stay as they are."""
import pytest
import torch

import exact_attention_37_gb300 as fa

from . import rules

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_attention_37_gb300 import build

    build.build()
    fa.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def alike(got, want):
    """The same numbers, but for the roundings of another form of the tanh."""
    assert bool(torch.isfinite(got).all())
    assert float((got.float() - want.float()).abs().max()) <= 2.0 ** -7 * max(1.0, float(want.float().abs().max()))


# gains: every score in the polynomial's range of a cap of 20, and some beyond it
@pytest.mark.parametrize("cap,gain", [(0.0, 1.0), (20.0, 1.0), (20.0, 12.0)])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("ids", [False, True])
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "bf16")])
@pytest.mark.parametrize("heads", [2, 160])
def test_a_query_and_a_key_that_are_nan(cap, gain, bias, ids, d, dtype, heads):
    N, bad = 300, 200
    q, k, v, do = rules.problem(d, dtype, 1, heads, heads, N, N, d, gain=gain)
    doc = rules.packed_ids([[150, 140]], pad=10) if ids else None
    rule = fa.ScoreRule(causal=True, cap=cap, slopes=rules.slopes(heads) if bias else None, q_doc=doc, k_doc=doc)
    ref = fa.forward_rule(q, k, v, rule)
    grads = fa.backward_rule(q, k, v, *ref, do, rule)
    end = 290 if ids else N  # rows 290 on are padding
    # a query: its own row only
    x = q.clone()
    x[:, 1, bad, 5] = NAN
    o, lse = fa.forward_rule(x, k, v, rule)
    assert bool(o[:, 1, bad].isnan().all()) and bool(lse[:, 1, bad].isnan().all())
    rest = torch.arange(N, device="cuda") != bad
    alike(o[:, :, rest], ref[0][:, :, rest])
    assert torch.equal(o[:, 0], ref[0][:, 0])
    dq, dk, dv = fa.backward_rule(x, k, v, o, lse, do, rule)
    sees = slice(150 if ids else 0, bad + 1)
    assert bool(dq[:, 1, bad].isnan().all()) and bool(dk[:, 1, sees].isnan().all()) and bool(dv[:, 1, sees].isnan().all())
    assert all(torch.equal(a[:, 0], b[:, 0]) for a, b in zip((dq, dk, dv), grads))
    # a key: the rows that see it
    x = k.clone()
    x[:, 1, bad, 5] = NAN
    o, lse = fa.forward_rule(q, x, v, rule)
    assert bool(o[:, 1, bad:end].isnan().all()) and bool(lse[:, 1, bad:end].isnan().all())
    alike(o[:, 1, :bad], ref[0][:, 1, :bad])
    dq, dk, dv = fa.backward_rule(q, x, v, o, lse, do, rule)
    assert bool(dq[:, 1, bad:end].isnan().all()) and bool(dv[:, 1, bad].isnan().all())
    fa.fa_check_device_status()


def test_rows_that_see_nothing_are_not_nan():
    q, k, v, _ = rules.problem(1, "bf16", 1, 2, 2, 300, 100, 64)
    o, lse = fa.forward_rule(q, k, v, fa.ScoreRule(causal=True, cap=5.0))
    assert bool((o[:, :, :200] == 0).all()) and bool((lse[:, :, :200] == -float("inf")).all())


# one CTA a sequence and clusters; stretches that are split, small and full grids; 8 parts and more
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B,H,Hkv,n,room", [(2, 4, 2, 90, 96), (2, 4, 2, 700, 704), (1, 4, 1, 700, 8000), (1, 4, 1, 8000, 8000),
                                            (3, 16, 4, 5000, 20000), (600, 2, 2, 40, 8192)])
def test_queries_over_a_cache(cap, dtype, B, H, Hkv, n, room):
    d, page = 128, 32
    g = torch.Generator().manual_seed(n)
    held = -(-n // page)
    cache = fa.KV4Cache.empty(held, Hkv, page, d, dtype)
    table = torch.zeros(B, -(-room // page), dtype=torch.int32)
    table[:, :held] = torch.arange(held)
    table = table.cuda()
    k, v = (torch.randn(1, Hkv, n, d, generator=g).to(dtype).cuda() for _ in range(2))
    fa.kv4_append(cache, k, v, table[:1].contiguous(), i32([0]))
    q = torch.randn(B, H, 1, d, generator=g).to(dtype).cuda()
    lens = i32([n] * B)
    ref = fa.kv4_attend(q, cache, table, lens, cap=cap)
    q[0, 1, 0, 7] = NAN
    o, lse = fa.kv4_attend(q, cache, table, lens, cap=cap)
    assert bool(o[0, 1].isnan().all()) and bool(lse[0, 1].isnan().all())
    o[0, 1], lse[0, 1] = ref[0][0, 1], ref[1][0, 1]
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    fa.fa_check_device_status()


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("n", [90, 700, 8000])
def test_a_cached_value_that_is_nan(cap, n):
    """One NaN in a token's key or value: the rows that attend over it."""
    d, page, dtype = 128, 32, torch.bfloat16
    g = torch.Generator().manual_seed(n)
    held = -(-n // page)
    table = torch.arange(held, dtype=torch.int32, device="cuda")[None]
    q = torch.randn(1, 4, 1, d, generator=g).to(dtype).cuda()
    for which in (0, 1):
        x = [torch.randn(1, 1, n, d, generator=g).to(dtype).cuda() for _ in range(2)]
        cache = fa.KV4Cache.empty(held, 1, page, d, dtype)
        fa.kv4_append(cache, *x, table, i32([0]))
        cache.pools[1 + 2 * which][(n - 20) // page, 0, (n - 20) % page, 1, 1] = NAN  # a group's low value
        o, lse = fa.kv4_attend(q, cache, table, i32([n]), cap=cap)
        if which == 0:
            assert bool(o.isnan().all()) and bool(lse.isnan().all())
        else:
            assert bool(o[..., 32:64].isnan().all())
            assert bool(torch.isfinite(o[..., :32]).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_stored_row_with_nan(dtype, d):
    """The smallest of a group with a NaN is NaN, and so is every value that it stands for."""
    n, page = 40, 16
    g = torch.Generator().manual_seed(d)
    k, v = (torch.randn(1, 2, n, d, generator=g).to(dtype) for _ in range(2))
    table = torch.arange(3, dtype=torch.int32, device="cuda")[None]

    def stored():
        cache = fa.KV4Cache.empty(3, 2, page, d, dtype)
        fa.kv4_append(cache, k.cuda(), v.cuda(), table, i32([0]))
        return fa.kv4_read(cache, table, i32([0]), n, i32([n]))

    ref = stored()
    at = [(0, 3, 0), (1, 17, 33), (1, 39, d - 1), (0, 8, 31)]
    for h, i, c in at:
        k[0, h, i, c] = NAN
        v[0, 1 - h, i, c] = -NAN
    for x, r, flip in zip(stored(), ref, (0, 1)):
        for h, i, c in at:
            part = (0, h ^ flip, i, slice(c // 32 * 32, c // 32 * 32 + 32))
            assert bool(x[part].isnan().all())
            x[part] = r[part]
        assert torch.equal(x, r)
