"""The 4-bit key/value cache written out from its definition (numpy and torch, float64
values).  Test infrastructure: nothing of it runs on the CUDA path."""
from __future__ import annotations

import numpy as np
import torch

GROUP = 32


def round_to(x: np.ndarray, dtype) -> np.ndarray:
    """float64 to the nearest value of fp16 or bf16 (ties to even), as float64; normal range."""
    if dtype == torch.float16:
        return x.astype(np.float16).astype(np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


def store(x: torch.Tensor):
    """Rows [..., d] of fp16 or bf16 to (codes [..., d], scale, low [..., d / 32]), every step in
    float32; codes as integers, scale and low as float64."""
    g = x.float().cpu().numpy().reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    low = g.min(-1)
    spread = (g.max(-1) - low).astype(np.float32)
    scale = torch.from_numpy(spread / np.float32(15)).to(x.dtype).float().numpy()
    scale = np.where(scale < np.float32(2.0 ** -126), np.float32(0), scale)
    with np.errstate(divide="ignore"):
        inv = np.where(scale > 0, np.float32(1) / scale, np.float32(0)).astype(np.float32)
    t = (g - low[..., None]).astype(np.float32) * inv[..., None]
    codes = np.minimum(15, np.rint(t)).astype(np.int64)
    return codes.reshape(*x.shape), scale.astype(np.float64), low.astype(np.float64)


def values(codes, scale, low, dtype) -> np.ndarray:
    """What codes stand for: T(low + scale * code), one rounding."""
    c = codes.reshape(*codes.shape[:-1], codes.shape[-1] // GROUP, GROUP).astype(np.float64)
    return round_to(low[..., None] + scale[..., None] * c, dtype).reshape(*codes.shape)


def cached(cache, which: str, pages, page_size: int, n: int) -> np.ndarray:
    """Values [H_kv, n, d] of the first n tokens of a sequence with the given pages."""
    codes = getattr(cache, which + "_codes").cpu().numpy()
    params = getattr(cache, which + "_params").double().cpu().numpy()
    H, d = codes.shape[1], 2 * codes.shape[3]
    c = np.zeros((H, n, d), np.int64)
    s, lo = np.zeros((H, n, d // GROUP)), np.zeros((H, n, d // GROUP))
    for p in range(n):
        page, r = pages[p // page_size], p % page_size
        c[:, p, 0::2], c[:, p, 1::2] = codes[page, :, r] & 15, codes[page, :, r] >> 4
        s[:, p], lo[:, p] = params[page, :, r, :, 0], params[page, :, r, :, 1]
    return values(c, s, lo, cache.dtype)


def attend(q, k, v, length, scale, causal=True, cap=0.0, slopes=None, hidden=()):
    """One sequence: q [H, N_q, d], k, v [H_kv, n, d] float64 -> (O, L, sum P |v|, sum |v|)."""
    H, Nq, d = q.shape
    g = H // k.shape[0]
    n = k.shape[1]
    o, a, z = np.zeros((H, Nq, d)), np.zeros((H, Nq, d)), np.zeros((H, Nq, d))
    lse = np.full((H, Nq), -np.inf)
    pos = length - Nq + np.arange(Nq)
    see = np.ones((Nq, n), bool)
    if causal:
        see = np.arange(n)[None] <= pos[:, None]
    see[:, list(hidden)] = False
    for h in range(H):
        y = scale * (q[h] @ k[h // g].T)
        if cap:
            y = cap * np.tanh(y / cap)
        if slopes is not None:
            y = y - slopes[h] * np.abs(pos[:, None] - np.arange(n)[None])
        for i in range(Nq):
            if not see[i].any():
                continue
            w = see[i]
            m = y[i, w].max()
            e = np.exp(y[i, w] - m)
            p = e / e.sum()
            lse[h, i] = m + np.log(e.sum())
            o[h, i], a[h, i], z[h, i] = p @ v[h // g][w], p @ np.abs(v[h // g][w]), np.abs(v[h // g][w]).sum(0)
    return o, lse, a, z
