"""CPU reference of the operators around a decode step's attention, numpy
float64 and whole numbers (test infrastructure).  Nothing here shares code
with the package.
"""

from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

# 1 / (2 pi), to 60 digits
_INV_2PI = Fraction("0.159154943091895335768883763372514362034459645740456448747667")
FAR = 64.0  # a token less likely than the likeliest by e^-64 is never drawn


# -------------------------------------------- queries and keys by position

def angles(positions, inv_freq):
    """cos, sin [T][n] of position * frequency, reduced in rational numbers."""
    turns = [[float(Fraction(float(f)) * int(p) * _INV_2PI % 1) for f in inv_freq]
             for p in positions]
    a = 2 * math.pi * np.array(turns, np.float64).reshape(len(positions), len(inv_freq))
    return np.cos(a), np.sin(a)


def rope(x, positions, inv_freq, layout, factor, weight, eps):
    """x float64 [T][H][D] -> (y, mag): the rotated heads, and |a| + |b| of each
    result's pair after the norm (times factor where it is turned)."""
    x = x.astype(np.float64)
    rot = 2 * len(inv_freq)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    y, mag = x.copy(), np.abs(x)
    cos, sin = angles(positions, inv_freq)
    for i in range(rot // 2):
        m, n = (i, rot // 2 + i) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = cos[:, i, None], sin[:, i, None]
        y[..., m] = factor * (x[..., m] * c - x[..., n] * s)
        y[..., n] = factor * (x[..., n] * c + x[..., m] * s)
        mag[..., m] = mag[..., n] = abs(factor) * (np.abs(x[..., m]) + np.abs(x[..., n]))
    return y, mag


# --------------------------------------------- the pages of a batch's tokens

def extend(table, lengths, refcount, rows, counts, total, page_size):
    """kv_pages_extend on lists, one request after the other; changes table,
    lengths and refcount, returns (status, starts, token_rows, positions)."""
    free = [p for p, c in enumerate(refcount) if c <= 0]
    status, starts, token_rows, positions = [], [0], [-1] * total, [-1] * total
    named, taken, sure, at = set(), 0, True, 0
    for row, count in zip(rows, counts):
        begin, at = at, at + max(count, 0)
        starts.append(min(at, total))
        ok = 0 <= row < len(table) and row not in named and count >= 0 and at <= total
        named.add(row)
        if ok:
            have = lengths[row]
            ok = have >= 0 and have + count <= len(table[row]) * page_size
        if not ok:
            status.append(2)
            continue
        old, new = -(-have // page_size), -(-(have + count) // page_size)
        sure = sure and taken + new - old <= len(free)
        taken += new - old
        if new > old and not sure:
            status.append(1)
            continue
        for i in range(old, new):
            table[row][i] = free[taken - new + i]
            refcount[table[row][i]] = 1
        lengths[row] = have + count
        status.append(0)
        for t in range(begin, at):
            token_rows[t], positions[t] = row, have + t - begin
    return status, starts, token_rows, positions


# --------------------------------------------------------- the next tokens

def sample(x, u, temperature, top_k, top_p, min_p):
    """(token, margin) of one row of logits float64 [V]: margin is how near the
    nearest decision was to its border, as a part of the mass it is about."""
    x = np.asarray(x, np.float64)
    if x.size == 0 or np.isnan(x).any() or x.max() in (math.inf, -math.inf) or temperature != temperature:
        return -1, 1.0
    if temperature <= 0:
        return int(np.argmax(x)), 1.0
    live = x > -math.inf
    z = np.where(live, np.where(live, x, 0.0) / temperature, -math.inf)
    d = np.where(live, z - z.max(), -math.inf).astype(np.longdouble)
    w = np.where(d > -FAR, np.exp(d), np.longdouble(0))
    order = np.lexsort((np.arange(x.size), -x))
    if 0 < top_k < x.size:
        order = order[:top_k]
    margin = 1.0
    if top_p < 1:
        mass = np.concatenate(([np.longdouble(0)], np.cumsum(w[order])))
        limit = np.longdouble(top_p) * mass[-1]
        n = max(1, int((mass[:-1] < limit).sum()))
        margin = min(margin, float(np.abs(mass[1:-1] - limit).min(initial=1.0) / mass[-1]))
        order = order[:n]
    if min_p > 0:
        least = np.longdouble(min(min_p, 1.0))
        if least < 1:
            margin = min(margin, float(np.abs(w[order] / least - 1).min()))
        order = order[w[order] >= least]
    kept = np.sort(order)
    mass = np.cumsum(w[kept])
    u = min(max(u, 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    target = np.longdouble(u) * mass[-1]
    if u > 0:
        margin = min(margin, float(np.abs(mass - target).min() / mass[-1]))
    i = int((mass <= target).sum())
    return int(kept[i]), margin
