"""CPU reference of the serving operators, numpy float64 (test infrastructure).

Plain definitions, one element or token at a time where that is the clearest
form; nothing here shares code with the package.
"""

from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------ 4-bit weights

def int4_dequant(codes, scales, zeros, group):
    """[N][K] float64 weight that codes, group scales and zero points stand for."""
    N, K = codes.shape
    w = np.empty((N, K))
    for k in range(K):
        g = k // group
        z = 8.0 if zeros is None else zeros[:, g].astype(np.float64)
        w[:, k] = (codes[:, k].astype(np.float64) - z) * scales[:, g].astype(np.float64)
    return w


def int4_quantize(W, group, symmetric):
    """(codes, scales float16, zeros or None): fp32 arithmetic, one rounding a step."""
    W = W.astype(np.float32)
    N, K = W.shape
    ng = -(-K // group)
    codes = np.zeros((N, K), np.uint8)
    scales = np.zeros((N, ng), np.float16)
    zeros = None if symmetric else np.zeros((N, ng), np.uint8)
    for g in range(ng):
        w = W[:, g * group:(g + 1) * group]
        lo = np.minimum(w.min(1), np.float32(0))
        hi = np.maximum(w.max(1), np.float32(0))
        span = np.maximum(hi, -lo) / np.float32(7) if symmetric else (hi - lo) / np.float32(15)
        s16 = np.minimum(span, np.float32(65504)).astype(np.float16)
        s = s16.astype(np.float32)
        d = np.where(s > 0, s, np.float32(1))
        if symmetric:
            z = np.full(N, 8, np.float32)
        else:
            z = np.where(s > 0, np.clip(np.rint(-lo / d), 0, 15), np.float32(0))
            zeros[:, g] = z.astype(np.uint8)
        q = np.clip(np.rint(w / d[:, None]) + z[:, None], 0, 15)
        q = np.where(s[:, None] > 0, q, z[:, None])
        codes[:, g * group:(g + 1) * group] = q.astype(np.uint8)
        scales[:, g] = s16
    return codes, scales, zeros


# -------------------------------------------------------- the paged cache

def kv_codes(x):
    """(codes int8, a) of float32 rows [..., dims]: a = max |x|, round half to even."""
    x = x.astype(np.float32)
    a = np.abs(x).max(-1)
    d = np.where(a > 0, a, np.float32(1))[..., None]
    q = np.clip(np.rint((np.float32(127) * x) / d), -127, 127)
    return np.where(a[..., None] > 0, q, 0).astype(np.int8), a


def attention_rows(q, k, v, scale, softcap):
    """One sequence and kv head: q [G][D], k, v [T][D] float64 -> out [G][D],
    lse [G], and eps-free sums for error bounds: sum p |v| [G][D], and the
    largest |scale| sum |q||k| of a row [G]."""
    G, D = q.shape
    T = k.shape[0]
    out, lse = np.zeros((G, D)), np.full(G, -math.inf)
    pv, mag = np.zeros((G, D)), np.zeros(G)
    if T == 0:
        return out, lse, pv, mag
    with np.errstate(all="ignore"):
        s = scale * (q @ k.T)
        if softcap > 0:
            s = softcap * np.tanh(s / softcap)
        mag = (abs(scale) * (np.abs(q) @ np.abs(k).T)).max(1)
        for g in range(G):
            m = s[g].max()
            if m == -math.inf:
                continue
            e = np.exp(s[g] - m)
            out[g] = (e / e.sum()) @ v
            pv[g] = (e / e.sum()) @ np.abs(v)
            lse[g] = m + math.log(e.sum()) if np.isfinite(e.sum()) else e.sum()
    return out, lse, pv, mag


# --------------------------------------------------------------- the pages

class Pool:
    """Tables, lengths and counts as Python lists, and what happens to pages as
    a list of (source, destination) copies."""

    def __init__(self, table, lengths, ref, page_size):
        self.table = [list(map(int, r)) for r in table]
        self.lengths = list(map(int, lengths))
        self.ref = list(map(int, ref))
        self.ps = page_size
        self.width = len(self.table[0]) if self.table else 0

    def _free_ids(self):
        return [i for i, r in enumerate(self.ref) if r <= 0]

    def free(self, rows):
        for r in rows:
            if not 0 <= r < len(self.table):
                continue
            for j, p in enumerate(self.table[r]):
                if 0 <= p < len(self.ref) and self.ref[p] > 0:
                    self.ref[p] -= 1
                self.table[r][j] = -1
            self.lengths[r] = 0

    def reserve(self, rows, new):
        free, status, out = self._free_ids(), [], False
        taken = 0
        for i, (r, n) in enumerate(zip(rows, new)):
            if not 0 <= r < len(self.table) or r in rows[:i] or self.lengths[r] < 0 or \
                    n < self.lengths[r] or n > self.width * self.ps:
                status.append(2)
                continue
            have = -(-self.lengths[r] // self.ps)
            need = -(-n // self.ps) - have
            if need and (out or taken + need > len(free)):
                out = True
                status.append(1)
                continue
            for j in range(need):
                page = free[taken + j]
                self.table[r][have + j] = page
                self.ref[page] = 1
            taken += need
            self.lengths[r] = n
            status.append(0)
        return status

    def fork(self, parents, children):
        """Status list; copies is the list of pages to copy."""
        free, status, copies = self._free_ids(), [], []
        taken = 0
        start = list(self.lengths)
        for i, (p, c) in enumerate(zip(parents, children)):
            S = len(self.table)
            ok = 0 <= p < S and 0 <= c < S and c not in children[:i] and p not in children
            ok = ok and start[c] == 0 and 0 <= start[p] <= self.width * self.ps
            whole, part = divmod(start[p], self.ps) if ok else (0, 0)
            if ok and part:
                ok = 0 <= self.table[p][whole] < len(self.ref)
            if not ok:
                status.append(2)
                continue
            if part and taken >= len(free):
                status.append(1)
                continue
            row = self.table[p][:whole]
            for page in row:
                if 0 <= page < len(self.ref):
                    self.ref[page] += 1
            if part:
                page = free[taken]
                taken += 1
                copies.append((self.table[p][whole], page))
                self.ref[page] = 1
                row = row + [page]
            self.table[c] = row + [-1] * (self.width - len(row))
            self.lengths[c] = start[p]
            status.append(0)
        return status, copies

    def compact(self):
        """(number of used pages, copies)."""
        P = len(self.ref)
        used = [r > 0 for r in self.ref]
        live = sum(used)
        holes = [i for i in range(live) if not used[i]]
        movers = [i for i in range(live, P) if used[i]]
        to = {m: h for m, h in zip(movers, holes)}
        for row in self.table:
            for j, p in enumerate(row):
                if not 0 <= p < P or (p >= live and p not in to):
                    row[j] = -1
                else:
                    row[j] = to.get(p, p)
        ref = [self.ref[i] if i < live and used[i] else 0 for i in range(P)]
        for m, h in to.items():
            ref[h] = self.ref[m]
        self.ref = ref
        return live, list(to.items())
