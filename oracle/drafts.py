"""Rotary positions, page tables and trees of drafted tokens written out from their definitions
(plain Python and numpy, float64 values).  Test infrastructure: nothing of it runs on the CUDA path."""
from __future__ import annotations

from decimal import Decimal, getcontext

import numpy as np

getcontext().prec = 80
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")


def turns(position: int, freq: float) -> float:
    """Fraction of a turn, in (-1/2, 1/2], of position * freq radians."""
    t = Decimal(position) * Decimal(freq) / TWO_PI
    return float(t - t.to_integral_value())


def rotary(x, positions, freqs, interleaved=False, amplitude=1.0, backward=False):
    """x [B, H, N, d] float64, positions [B, N], freqs [dims / 2] -> (y, |x1| + |x2| of each channel's pair)."""
    half = len(freqs)
    table = {}
    for p in {int(v) for v in positions.reshape(-1)}:
        table[p] = np.array([turns(p, float(f)) for f in freqs])
    t = 2 * np.pi * np.stack([[table[int(p)] for p in row] for row in positions])[:, None]  # [B, 1, N, half]
    cos, sin = amplitude * np.cos(t), amplitude * np.sin(-t if backward else t)
    first = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
    second = first + 1 if interleaved else first + half
    y, size = x.copy(), np.zeros_like(x)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    size[..., first] = size[..., second] = np.abs(a) + np.abs(b)
    return y, size


def ancestors(parents, count, prefix):
    """For each drafted token the list of itself and its ancestors, the oldest first; None for one that is no token
    of the tree."""
    out = []
    for i, p in enumerate(parents):
        if i >= count or prefix + i < 0 or p < -1 or p >= i or (p >= 0 and out[p] is None):
            out.append(None)
        else:
            out.append(([] if p < 0 else out[p]) + [i])
    return out


def attend_tree(q, k, v, parents, count, length, scale, cap=0.0, slopes=None, hidden=()):
    """One sequence: q [H, N_q, d], k, v [H_kv, length, d] float64 -> (O, L, sum P |v|, sum |v| of the seen)."""
    H, Nq, d = q.shape
    g = H // k.shape[0]
    m = min(max(count, 0), Nq)
    prefix = length - m
    rows = ancestors(parents, m, prefix)
    o, a, z = np.zeros((H, Nq, d)), np.zeros((H, Nq, d)), np.zeros((H, Nq, d))
    lse = np.full((H, Nq), -np.inf)
    pos = np.arange(length, dtype=np.float64)
    for i in range(m):
        if prefix + i >= 0:
            pos[prefix + i] = prefix + (len(rows[i]) - 1 if rows[i] else 0)
    for i in range(Nq):
        if rows[i] is None:
            continue
        see = np.array([t for t in list(range(max(prefix, 0))) + [prefix + j for j in rows[i]] if t not in hidden], dtype=int)
        if not len(see):
            continue
        for h in range(H):
            kk, vv = k[h // g][see], v[h // g][see]
            y = scale * (kk @ q[h, i])
            if cap:
                y = cap * np.tanh(y / cap)
            if slopes is not None:
                y = y - slopes[h] * np.abs(prefix + len(rows[i]) - 1 - pos[see])
            top = y.max()
            e = np.exp(y - top)
            p = e / e.sum()
            lse[h, i] = top + np.log(e.sum())
            o[h, i], a[h, i], z[h, i] = p @ vv, p @ np.abs(vv), np.abs(vv).sum(0)
    return o, lse, a, z


def plan(table, held, free, free_count, page, start, count, N, parents=None):
    """fa_kv4_plan on lists: (table, held, free, free_count, out_count, lengths, slots, positions)."""
    table, held, free = [list(r) for r in table], list(held), list(free)
    B, room = len(table), len(table[0]) if table else 0
    start = [max(s, 0) for s in start]
    count = [min(max(c, 0), N) for c in count]
    held = [min(max(h, 0), room) for h in held]
    top = min(max(free_count, 0), len(free))
    want = [-(-(s + c) // page) for s, c in zip(start, count)]
    for b in reversed(range(B)):
        if want[b] < held[b]:
            for p in reversed(range(want[b], held[b])):
                free[top] = table[b][p]
                table[b][p] = -1
                top += 1
            held[b] = want[b]
    out, stopped = [], False
    for b in range(B):
        more = want[b] - held[b]
        if want[b] > room:
            out.append(0)
            continue
        if more > 0:
            stopped = stopped or more > top
            if stopped:
                out.append(0)
                continue
            for p in range(held[b], want[b]):
                top -= 1
                table[b][p] = free[top]
            held[b] = want[b]
        out.append(count[b])
    lengths = [s + c for s, c in zip(start, out)]
    slots, positions = [], []
    for b in range(B):
        rows = ancestors(parents[b], out[b], 0) if parents is not None else None
        sl, po = [], []
        for i in range(N):
            t = start[b] + i
            if i >= out[b]:
                sl.append(-1)
                po.append(-1)
                continue
            e = table[b][t // page]
            sl.append(-1 if e < 0 else e * page + t % page)
            po.append(t if rows is None else -1 if rows[i] is None else start[b] + len(rows[i]) - 1)
        slots.append(sl)
        positions.append(po)
    return table, held, free, top, out, lengths, slots, positions
