"""Inputs of the tests of drafted tokens."""
import numpy as np
import torch


def i32(x, device="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=device)


def tree(rng, N, roots=0.15):
    """Parents of N drafted tokens: a random tree, some hanging off the prefix."""
    return [-1 if i == 0 or rng.random() < roots else int(rng.integers(max(0, i - 6), i)) for i in range(N)]


def chain(N):
    return list(range(-1, N - 1))


def bounds():
    """Half steps of the types: of a rounding, and of fp16's smallest numbers."""
    return {torch.float16: (2.0 ** -11, 2.0 ** -25), torch.bfloat16: (2.0 ** -8, 2.0 ** -134)}


def over_bound(got, want, weight, seen, t):
    """Attention's O against its bound (as for the other kernels): u (sum P |v| + |O|) + 1e-4 sum P |v| + s (sum |v| + 1)."""
    u, s = bounds()[t]
    return (np.abs(got - want) / (u * (weight + np.abs(want)) + 1e-4 * weight + s * (seen + 1))).max()
