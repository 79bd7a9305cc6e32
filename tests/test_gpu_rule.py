"""Attention with a score rule on the GPU against the float64 definition: caps, distance
bias, document ids, prefixes and their combinations, forward and backward."""
import pytest
import torch

import exact_attention_37_gb300 as fa
from oracle import rules as oracle

from . import rules

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_attention_37_gb300 import build

    build.build()
    fa.load()


def ids_of(kind, B, N):
    """Document ids [B, N] of a kind, or None."""
    if kind is None:
        return None
    g = torch.Generator().manual_seed(N + B)
    if kind == "packed":  # consecutive documents, one of a single row, padding behind
        cut = torch.sort(torch.randint(0, N, (B, 3), generator=g), 1)[0]
        x = (torch.arange(N)[None, :, None] >= cut[:, None, :]).sum(-1)
        x[:, N - N // 7:] = -1
    elif kind == "mixed":  # any ids in any order, negative ones among them
        x = torch.randint(-2, 4, (B, N), generator=g)
    elif kind == "one":    # one document: everything is seen in full
        x = torch.full((B, N), 7)
    elif kind == "none":   # nothing is seen by anything
        x = torch.full((B, N), -5)
    elif kind == "large":  # ids at the ends of the type
        x = torch.where(torch.arange(N)[None] % 2 == 0, 2 ** 31 - 1, -2 ** 31).expand(B, N)
    return x.to(torch.int32).contiguous().cuda()


RULES = [  # causal, cap, bias, ids, prefix
    (False, 0.0, False, None, 0),
    (True, 0.0, False, None, 70),
    (True, 30.0, False, None, 0),
    (False, 2.0, True, None, 0),
    (True, 0.0, True, None, 200),
    (False, 0.0, True, None, 0),
    (True, 0.0, False, "packed", 0),
    (True, 50.0, True, "packed", 40),
    (False, 4.0, False, "mixed", 0),
    (True, 0.0, True, "mixed", 0),
    (True, 0.0, False, "one", 0),
    (True, 10.0, False, "none", 0),
    (False, 0.0, False, "large", 0),
]


def make_rule(r, B, H, Nq, Nk):
    causal, cap, bias, kind, prefix = r
    ids = ids_of(kind, B, max(Nq, Nk))
    q_doc = ids[:, max(Nq, Nk) - Nq:].contiguous() if ids is not None else None
    k_doc = ids[:, max(Nq, Nk) - Nk:].contiguous() if ids is not None else None
    pre = torch.tensor([prefix + 9 * b for b in range(B)], dtype=torch.int32, device="cuda") if prefix else None
    return fa.ScoreRule(causal=causal, cap=cap, slopes=rules.slopes(H) if bias else None, q_doc=q_doc, k_doc=k_doc,
                        prefix=pre)


@pytest.mark.parametrize("r", RULES, ids=str)
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "bf16")])
def test_forward_every_rule(r, d, dtype):
    B, H, Hkv, Nq, Nk = 2, 4, 2, 300, 300
    q, k, v, _ = rules.problem(d, dtype, B, H, Hkv, Nq, Nk, d, gain=3.0 if r[1] else 1.0)
    rules.check_forward(q, k, v, make_rule(r, B, H, Nq, Nk))


@pytest.mark.parametrize("r", RULES, ids=str)
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "bf16")])
def test_backward_every_rule(r, d, dtype):
    B, H, Hkv, Nq, Nk = 2, 4, 2, 300, 300
    q, k, v, do = rules.problem(1000 + d, dtype, B, H, Hkv, Nq, Nk, d, gain=3.0 if r[1] else 1.0)
    rules.check_backward(q, k, v, do, make_rule(r, B, H, Nq, Nk))


@pytest.mark.parametrize("Nq,Nk", [(1, 1), (1, 700), (129, 128), (128, 257), (500, 260), (3, 1000), (641, 641)])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16"), (256, "fp16")])
def test_lengths(Nq, Nk, d, dtype):
    """From one row on, more keys than queries and fewer, block edges."""
    B, H, Hkv = 1, 3, 1
    q, k, v, do = rules.problem(Nq + Nk + d, dtype, B, H, Hkv, Nq, Nk, d, gain=2.0)
    for r in ((True, 20.0, True, None, 5), (True, 0.0, False, "packed", 0), (False, 20.0, True, "mixed", 0)):
        rules.check_backward(q, k, v, do, make_rule(r, B, H, Nq, Nk))
        rules.check_forward(q, k, v, make_rule(r, B, H, Nq, Nk))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_grids_take_the_256_row_blocks(d):
    """Enough heads for two sub-tiles a CTA; documents that end inside both."""
    B, H, Hkv, N = 4, 40, 8, 530
    q, k, v, do = rules.problem(77 + d, "bf16", B, H, Hkv, N, N, d, gain=2.0)
    for r in ((True, 25.0, True, "packed", 33), (True, 0.0, False, "mixed", 0), (True, 0.0, True, None, 300),
              (True, 3.0, False, None, 0)):
        rules.check_backward(q, k, v, do, make_rule(r, B, H, N, N))
        rules.check_forward(q, k, v, make_rule(r, B, H, N, N))


@pytest.mark.parametrize("cap", [0.05, 1.0, 1000.0, 1e6])
def test_caps_from_saturated_to_almost_none(cap):
    q, k, v, do = rules.problem(5, "bf16", 1, 4, 4, 260, 260, 64, gain=3.0)
    rules.check_backward(q, k, v, do, fa.ScoreRule(causal=True, cap=cap))
    rules.check_forward(q, k, v, fa.ScoreRule(causal=True, cap=cap))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 65504.0])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", [3, 200])
def test_padding_rows_may_hold_anything(bad, cap, d, heads):
    """Rows with a negative id are not used, whatever Q, K, V, O and dO hold there.  Without a
    cap the results are the same to the bit.  With one, a warp takes one of two forms of the
    tanh by the scores of its chunk, unused ones among them, so what the padding holds may
    change the form: both are within the bounds, which is what holds then."""
    B, N = 1, 400 if heads == 3 else 300
    q, k, v, do = rules.problem(31 + d, "fp16", B, heads, heads, N, N, d)
    ids = rules.packed_ids([[90, 130, N - 250]], pad=30)
    ids[:, 17:20] = -1  # padding inside a document too
    pad = (ids < 0)[0]
    rule = fa.ScoreRule(causal=True, cap=cap, q_doc=ids, k_doc=ids)
    o, lse = fa.forward_rule(q, k, v, rule)
    ref = fa.backward_rule(q, k, v, o, lse, do, rule)
    for t in (q, k, v, do):
        t[:, :, pad] = bad
    o2, lse2 = rules.check_forward(q, k, v, rule)
    assert bool((o2[:, :, pad] == 0).all()) and bool((lse2[:, :, pad] == -float("inf")).all())
    if cap == 0:
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _, _, got = rules.check_backward(q, k, v, do, rule)
    for b in got:
        assert bool((b[:, :, pad] == 0).all())
    o2[:, :, pad] = bad
    again = fa.backward_rule(q, k, v, o2, lse2, do, rule)
    fa.fa_check_device_status()
    for a, b, c in zip(ref, got, again):
        assert torch.equal(b, c)
        if cap == 0:
            assert torch.equal(a, b)


def test_the_mask_alone_gives_the_plain_call():
    q, k, v, do = rules.problem(3, "bf16", 2, 4, 2, 700, 900, 128)
    for causal in (False, True):
        o, lse = fa.forward(q, k, v, causal=causal)
        ro, rl = fa.forward_rule(q, k, v, fa.ScoreRule(causal=causal))
        assert torch.equal(o, ro) and torch.equal(lse, rl)
        for a, b in zip(fa.backward(q, k, v, o, lse, do, causal=causal),
                        fa.backward_rule(q, k, v, o, lse, do, fa.ScoreRule(causal=causal))):
            assert torch.equal(a, b)


@pytest.mark.parametrize("cap,gain", [(6e4, 40.0), (2e5, 40.0), (1e7, 40.0), (1e14, 3.0)])
def test_caps_whose_polynomial_has_fewer_terms(cap, gain):
    """scale / cap from 2e-6 down: a cap that is none in all but name."""
    q, k, v, do = rules.problem(6, "bf16", 1, 2, 2, 200, 200, 64, gain=gain)
    rules.check_forward(q, k, v, fa.ScoreRule(causal=True, cap=cap))


@pytest.mark.parametrize("kind", [None, "packed", "mixed"])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16"), (256, "bf16")])
def test_prefixes_outside_the_keys_and_without_the_mask(kind, d, dtype):
    """Clipped to the keys under the causal mask; without it they change nothing."""
    B, H, N = 2, 4, 330
    q, k, v, do = rules.problem(d, dtype, B, H, 2, N, N, d)
    ids = ids_of(kind, B, N)
    pre = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def step(causal, prefix):
        rule = fa.ScoreRule(causal=causal, q_doc=ids, k_doc=ids, prefix=prefix)
        o, lse = fa.forward_rule(q, k, v, rule)
        return (o, lse, *fa.backward_rule(q, k, v, o, lse, do, rule))

    for causal, a, b in ((True, pre(-7, N + 1000), pre(0, N)), (True, pre(-2 ** 31, 2 ** 31 - 1), pre(0, N)), (True, pre(0, 0), None),
                         (False, pre(50, 200), None), (False, pre(-1, 2 ** 31 - 1), None)):
        for x, y in zip(step(causal, a), step(causal, b)):
            assert torch.equal(x, y)
    fa.fa_check_device_status()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "bf16")])
def test_slopes_of_either_sign(causal, d, dtype):
    """A negative slope favours far keys; one of 0 beside a steep one.

    Some keys are seen with a P below 2^-126 only, which the fp32 exponential gives as 0 (it
    flushes what is not a normal number): each visible pair's P is off by up to 2^-126, and its
    dS by that times |dP - D| <= top, so the gradients by 2^-126 (1 + top) of the sums of the
    other factors, next to the bounds of rules.py."""
    B, H, N = 1, 4, 500
    q, k, v, do = rules.problem(d, dtype, B, H, 4, N, N, d)
    rule = fa.ScoreRule(causal=causal, cap=30.0, slopes=torch.tensor([-0.02, 0.0, 4.0, -0.3], device="cuda"))
    o, lse = rules.check_forward(q, k, v, rule)
    scale = rules.f32(d ** -0.5)
    grads = fa.backward_rule(q, k, v, o, lse, do, rule, scale=scale)
    fa.fa_check_device_status()
    ref, mag, back, last = oracle.backward(q, k, v, o, lse, do, scale, **rules.kwargs(rule))
    u, s = rules.U[q.dtype], rules.S[q.dtype]
    top = d * float(do.abs().max()) * (float(v.abs().max()) + float(o.abs().max()))
    for n, g, r, m, w, x in zip(("dQ", "dK", "dV"), grads, ref, mag, back, last):
        rules.within(g, r, u * (m + r.abs()) + rules.E * (m + w / 16) + (s + 2.0 ** -126 * (1 + top)) * (x + 1), n)
