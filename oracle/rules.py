"""Attention with a score rule, written out from its definition in float64 (torch, any device).

Test infrastructure like the rest of this package: nothing of it runs on the CUDA path.

    u = scale q_i.k_j,  z = cap tanh(u / cap) (u without a cap),  y = z - slope_h |p_i - j|,
    p_i = i + N_k - N_q;  visible: ids equal and not negative, and (not causal, or j <= p_i,
    or j < prefix).  Rows with a negative id are not used, whatever they hold.

Besides the results each function returns the sums of absolute terms that a bound on
rounding errors needs.
"""
from __future__ import annotations

import torch


def clean(x, ids):
    """Rows with a negative id become zero ([B, H, N, d] and ids [B, N] or None)."""
    x = x.double()
    return x if ids is None else torch.where((ids >= 0)[:, None, :, None], x, torch.zeros_like(x))


def visible(B, Nq, Nk, causal, q_doc, k_doc, prefix, device):
    p = torch.arange(Nq, device=device)[:, None] + Nk - Nq
    j = torch.arange(Nk, device=device)[None, :]
    see = torch.ones(B, Nq, Nk, dtype=torch.bool, device=device)
    if causal:
        see &= j <= p
        if prefix is not None:
            see = see | (j[None] < prefix[:, None, None])
    if q_doc is not None:
        see &= (q_doc[:, :, None] == k_doc[:, None, :]) & (k_doc[:, None, :] >= 0)
    return see


def _scores(q, k, scale, cap, slopes, b, h, hk):
    u = scale * (q[b, h] @ k[b, hk].T)
    t = torch.tanh(u / cap) if cap else None
    y = cap * t if cap else u
    if slopes is not None:
        Nq, Nk = u.shape
        p = torch.arange(Nq, device=u.device)[:, None] + Nk - Nq
        y = y - slopes[h].double() * (p - torch.arange(Nk, device=u.device)[None]).abs()
    return y, (1 - t * t if cap else torch.ones_like(u))


def forward(q, k, v, scale, causal=False, cap=0.0, slopes=None, q_doc=None, k_doc=None, prefix=None):
    """(O, L, sum_j P |v|, sum over the visible j of |v|)."""
    q, k, v = clean(q, q_doc), clean(k, k_doc), clean(v, k_doc)
    B, H, Nq, d = q.shape
    g = H // k.shape[1]
    see = visible(B, Nq, k.shape[2], causal, q_doc, k_doc, prefix, q.device)
    o, a, n = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.zeros(B, H, Nq, dtype=torch.float64, device=q.device)
    for b in range(B):
        for h in range(H):
            y, _ = _scores(q, k, scale, cap, slopes, b, h, h // g)
            y = torch.where(see[b], y, torch.full_like(y, -torch.inf))
            m = y.max(-1, keepdim=True)[0].clamp(min=-1e300)
            e = torch.exp(y - m)
            s = e.sum(-1, keepdim=True)
            p = torch.where(s > 0, e / s.clamp(min=1e-300), torch.zeros_like(e))
            lse[b, h] = torch.where(s > 0, m + torch.log(s.clamp(min=1e-300)), torch.full_like(s, -torch.inf))[:, 0]
            o[b, h], a[b, h], n[b, h] = p @ v[b, h // g], p @ v[b, h // g].abs(), see[b].double() @ v[b, h // g].abs()
    return o, lse, a, n


def backward(q, k, v, o, lse, dout, scale, causal=False, cap=0.0, slopes=None, q_doc=None, k_doc=None, prefix=None):
    """((dQ, dK, dV), the same sums over absolute terms, and the sums that the differences
    dP - D put behind them, the sums of the last factor alone over the visible pairs) for the given O and L."""
    q, k, v = clean(q, q_doc), clean(k, k_doc), clean(v, k_doc)
    o, dout = clean(o, q_doc), clean(dout, q_doc)
    B, H, Nq, d = q.shape
    g = H // k.shape[1]
    see = visible(B, Nq, k.shape[2], causal, q_doc, k_doc, prefix, q.device)
    out = [torch.zeros_like(x) for x in (q, k, v)]
    mag = [torch.zeros_like(x) for x in (q, k, v)]
    back = [torch.zeros_like(x) for x in (q, k, v)]
    last = [torch.zeros_like(x) for x in (q, k, v)]
    for b in range(B):
        for h in range(H):
            hk = h // g
            y, f = _scores(q, k, scale, cap, slopes, b, h, hk)
            l = lse[b, h].double()[:, None]
            p = torch.where(see[b], torch.exp(y - torch.where(torch.isinf(l), torch.zeros_like(l), l)), torch.zeros_like(y))
            dp, D = dout[b, h] @ v[b, hk].T, (dout[b, h] * o[b, h]).sum(-1, keepdim=True)
            du = p * (dp - D) * f * scale
            out[0][b, h], mag[0][b, h] = du @ k[b, hk], du.abs() @ k[b, hk].abs()
            out[1][b, hk] += du.T @ q[b, h]
            mag[1][b, hk] += du.abs().T @ q[b, h].abs()
            out[2][b, hk] += p.T @ dout[b, h]
            mag[2][b, hk] += p.T @ dout[b, h].abs()
            w = p * (dout[b, h].abs() @ v[b, hk].abs().T + (dout[b, h] * o[b, h]).abs().sum(-1, keepdim=True)) * scale
            back[0][b, h] = w @ k[b, hk].abs()
            back[1][b, hk] += w.T @ q[b, h].abs()
            n = see[b].double()
            last[0][b, h] = scale * (n @ k[b, hk].abs())
            last[1][b, hk] += scale * (n.T @ q[b, h].abs())
            last[2][b, hk] += n.T @ dout[b, h].abs()
    return tuple(out), tuple(mag), tuple(back), tuple(last)
