"""Plain forms of the block tables and of the rotary positions: one request, one row after the
other.  Nothing here calls the library."""
from __future__ import annotations

import math

import numpy as np


def up(x, ps):
    return -(-x // ps)


def reserve(table, lens, free, n_free, new, ps):
    """Lists, changed in place; returns (n_free, starts, counts)."""
    most = len(table[0]) * ps
    starts, counts, wanted, left = [], [], 0, n_free
    for b, n in enumerate(new):
        n = max(n, 0)
        starts.append(lens[b])
        need = up(lens[b] + n, ps) - up(lens[b], ps)
        if lens[b] + n > most:
            counts.append(0)
            continue
        wanted += need
        if need and wanted > n_free:
            counts.append(0)
            continue
        for j in range(up(lens[b], ps), up(lens[b] + n, ps)):
            left -= 1
            table[b][j] = free[left]
        lens[b] += n
        counts.append(n)
    return left, starts, counts


def release(table, lens, free, n_free, keep, ps, pinned=None):
    for b, k in enumerate(keep):
        k = min(lens[b], max(k, 0))
        for j in range(up(k, ps), up(lens[b], ps)):
            if pinned is None or j >= pinned[b]:
                free[n_free] = table[b][j]
                n_free += 1
            table[b][j] = -1
        lens[b] = k
    return n_free


def slots(table, starts, counts, ps):
    """[(position, slot)] of every new token, by sequence."""
    return [[(s + i, table[b][(s + i) // ps] * ps + (s + i) % ps) for i in range(c)]
            for b, (s, c) in enumerate(zip(starts, counts))]


def inv_freq(rot, base=10000.0, scaling=None, factor=1.0, original=0, fast=32.0, slow=1.0):
    """(radians a token of each pair, amplitude), extended precision where the machine has it."""
    L = np.longdouble
    i = np.arange(rot // 2, dtype=L)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = np.exp(-2 * i / rot * np.log(L(base)))
    if scaling == "linear":
        return f / L(factor), 1.0
    if scaling == "parts":
        def at(turns):
            return rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
        r = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return f * (1 - r) + f / L(factor) * r, 0.1 * math.log(factor) + 1
    return f, 1.0


def turned(x, positions, freq, amplitude, interleaved, inverse=False):
    """fp64 rows [B, heads, N, d] turned by positions [B, N]."""
    rot = 2 * len(freq)
    turns = positions.astype(np.longdouble)[:, None, :, None] * (freq / (2 * np.longdouble(np.pi)))
    angle = ((turns - np.floor(turns)) * (2 * np.longdouble(np.pi))).astype(np.float64)
    c, s = amplitude * np.cos(angle), amplitude * np.sin(angle)
    if inverse:
        s = -s
    y = x.copy()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def partner(x, rot, interleaved):
    """|a| + |b| of the pair that each value belongs to (0 past rot)."""
    y = np.zeros_like(x)
    if interleaved:
        s = np.abs(x[..., 0:rot:2]) + np.abs(x[..., 1:rot:2])
        y[..., 0:rot:2] = y[..., 1:rot:2] = s
    else:
        s = np.abs(x[..., :rot // 2]) + np.abs(x[..., rot // 2:rot])
        y[..., :rot // 2] = y[..., rot // 2:rot] = s
    return y
