"""Helpers of the score-rule tests: seeded problems, the CUDA path, and bounds.

Bounds, with u the largest relative error of one rounding to the 16-bit type (finfo.eps / 2)
and E = 1e-4 for everything in fp32 (sums of up to some thousand terms, ex2, the tanh):
  O  : P and O are rounded once each:          u (sum P |v| + |O|) + E sum P |v|
  dV : P and dV:                               u (sum P |dO| + |dV|) + E sum P |dO|
  dQ : dS and dQ:  u (scale sum |dS| |k| + |dQ|) + E scale sum (|dS| + P sum(|dO||v| + |dO||O|) / 16) |k|
       (dP - D is a difference of fp32 sums whose errors are relative to their terms; 1e-4 / 16
        of them is about 2^-17, above d 2^-24 for d = 256 taken once)
  dK : as dQ with q for k
  L  : 3e-5 max(1, |L|)
plus, with S half of the type's smallest step (2^-25 for fp16; bf16 reaches as far down as
fp32): a P or dS below 2^-14 is rounded to fp16 with an absolute error of up to S, so each
visible pair adds S times its other factor (|v|, |dO|, scale |k|, scale |q|), and the result
itself is off by up to S more.  (In the forward pass P is at most 1 over a row sum of at
least 1, so S bounds the error of P over the row sum too.)
"""
from __future__ import annotations

import torch

import exact_attention_37_gb300 as fa
from oracle import rules as oracle

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
S = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
E = 1e-4


def problem(seed, dtype, B, H, Hkv, Nq, Nk, d, gain=1.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = TYPES[dtype]
    return [x.to(t).to(device) for x in (gain * r(B, H, Nq, d), r(B, Hkv, Nk, d), r(B, Hkv, Nk, d), r(B, H, Nq, d))]


def slopes(H, device="cuda"):
    return torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H).to(device)


def packed_ids(lengths, pad=0, device="cuda"):
    """[B, N] ids of consecutive documents and padding behind them; one list of lengths a row."""
    rows = [sum(([i] * n for i, n in enumerate(ls)), []) + [-1] * pad for ls in lengths]
    return torch.tensor(rows, dtype=torch.int32, device=device)


def f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def kwargs(rule):
    return dict(causal=rule.causal, cap=f32(rule.cap), slopes=rule.slopes, q_doc=rule.q_doc, k_doc=rule.k_doc,
                prefix=rule.prefix)


def within(got, ref, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got - ref).abs() / (bound + 1e-300)).max() if ref.numel() else torch.zeros(())
    assert float(over) <= 1.0, f"{what}: {float(over):.3g} of its bound"
    return float(over)


def check_l(lse, ref, what="L"):
    inf = torch.isinf(ref)
    assert torch.equal(torch.isinf(lse), inf) and bool((lse[inf] < 0).all()), f"{what}: rows that see nothing differ"
    err = (lse.double() - ref)[~inf].abs() / ref[~inf].abs().clamp(min=1.0)
    assert err.numel() == 0 or float(err.max()) <= 3e-5, f"{what}: {float(err.max()):.3g}"


def check_forward(q, k, v, rule, scale=None):
    scale = f32(q.shape[-1] ** -0.5 if scale is None else scale)
    o, lse = fa.forward_rule(q, k, v, rule, scale=scale)
    fa.fa_check_device_status()
    ro, rl, a, n = oracle.forward(q, k, v, scale, **kwargs(rule))
    u, s = U[q.dtype], S[q.dtype]
    within(o, ro, u * (a + ro.abs()) + E * a + s * (n + 1), "O")
    check_l(lse, rl)
    return o, lse


def check_backward(q, k, v, do, rule, scale=None):
    scale = f32(q.shape[-1] ** -0.5 if scale is None else scale)
    o, lse = fa.forward_rule(q, k, v, rule, scale=scale)
    grads = fa.backward_rule(q, k, v, o, lse, do, rule, scale=scale)
    fa.fa_check_device_status()
    ref, mag, back, last = oracle.backward(q, k, v, o, lse, do, scale, **kwargs(rule))
    u, s = U[q.dtype], S[q.dtype]
    for n, g, r, m, w, x in zip(("dQ", "dK", "dV"), grads, ref, mag, back, last):
        within(g, r, u * (m + r.abs()) + E * (m + w / 16) + s * (x + 1), n)
    return o, lse, grads
