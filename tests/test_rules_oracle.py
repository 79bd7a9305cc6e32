"""The float64 definition of attention with a score rule: its gradient against central
differences, and its special cases against the plain oracle."""
import numpy as np
import pytest
import torch

import oracle as plain
from oracle import rules


def inputs(B=2, H=4, Hkv=2, Nq=7, Nk=9, d=5, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return r(B, H, Nq, d), r(B, Hkv, Nk, d), r(B, Hkv, Nk, d), r(B, H, Nq, d)


RULE = dict(causal=True, cap=1.5, slopes=torch.tensor([0.5, 0.25, 0.1, 0.0]),
            q_doc=torch.tensor([[0, 0, 1, 1, 1, -1, 2], [3, 3, 3, 3, 3, 3, 3]], dtype=torch.int32),
            k_doc=torch.tensor([[0, 0, 0, 1, 1, 1, 1, -1, 2], [3, 3, 3, 4, 3, 3, 3, 3, 3]], dtype=torch.int32),
            prefix=torch.tensor([4, 0], dtype=torch.int32))


@pytest.mark.parametrize("drop", [(), ("cap",), ("slopes",), ("q_doc", "k_doc"), ("prefix",), ("causal",)])
def test_gradient_against_differences(drop):
    rule = {k: v for k, v in RULE.items() if k not in drop}
    q, k, v, do = inputs()
    o, lse, _, _ = rules.forward(q, k, v, 0.4, **rule)
    grads, _, _, _ = rules.backward(q, k, v, o, lse, do, 0.4, **rule)
    loss = lambda *x: float((rules.forward(*x, 0.4, **rule)[0] * rules.clean(do, rule.get("q_doc"))).sum())  # noqa: E731
    g = torch.Generator().manual_seed(1)
    for n in range(3):
        for _ in range(25):
            i = tuple(int(torch.randint(0, s, (1,), generator=g)) for s in (q, k, v)[n].shape)
            x = [q.clone(), k.clone(), v.clone()]
            h = 1e-5
            x[n][i] += h
            up = loss(*x)
            x[n][i] -= 2 * h
            # central differences: error about h^2 times a third derivative of order 1, and 1e-16 / h
            assert abs((up - loss(*x)) / (2 * h) - float(grads[n][i])) < 1e-7


@pytest.mark.parametrize("causal", [False, True])
def test_without_a_rule_it_is_plain_attention(causal):
    q, k, v, do = inputs(Nq=9)
    o, lse, _, _ = rules.forward(q, k, v, 0.3, causal=causal)
    kk, vv = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    n = [x.numpy() for x in (q, kk, vv, do)]  # (torch tensors would pass through 32 bits there)
    ro, rl = plain.attention_forward(*n[:3], 0.3, causal)
    assert np.abs(o.numpy() - ro).max() < 1e-12 and np.abs(lse.numpy() - rl).max() < 1e-12
    rdq, _, _, _ = plain.attention_backward(*n, 0.3, causal)
    (dq, _, _), _, _, _ = rules.backward(q, k, v, o, lse, do, 0.3, causal=causal)
    assert np.abs(dq.numpy() - rdq).max() < 1e-12


def test_what_each_part_does():
    q, k, v, _ = inputs(B=1, H=1, Hkv=1, Nq=6, Nk=6)
    base = rules.forward(q, k, v, 1.0)[0]
    assert not torch.allclose(base, rules.forward(q, k, v, 1.0, cap=0.5)[0])
    # a cap far above every score changes nothing, a very steep bias leaves the row's own key
    assert torch.allclose(base, rules.forward(q, k, v, 1.0, cap=1e9)[0], atol=1e-9)
    assert torch.allclose(rules.forward(q, k, v, 1.0, slopes=torch.tensor([1e4]))[0], v, atol=1e-12)
    # a prefix as long as the keys undoes the causal mask
    assert torch.allclose(base, rules.forward(q, k, v, 1.0, causal=True, prefix=torch.tensor([6]))[0], atol=1e-12)
    # documents of one row each leave the row's own key; padding sees nothing
    ids = torch.tensor([[0, 1, 2, 3, 4, -1]], dtype=torch.int32)
    o, lse, _, _ = rules.forward(q, k, v, 1.0, q_doc=ids, k_doc=ids)
    assert torch.allclose(o[0, 0, :5], v[0, 0, :5], atol=1e-12)
    assert bool((o[0, 0, 5] == 0).all()) and float(lse[0, 0, 5]) == -float("inf")
