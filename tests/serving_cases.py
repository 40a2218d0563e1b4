"""Inputs and comparisons shared by the GPU tests of the serving operators.

Unit roundoffs: u16 is half a unit of the result's type in the last place
(2^-11 float16, 2^-8 bfloat16; the results' one rounding), u32 = 2^-24."""

import numpy as np
import torch

U32 = 2.0 ** -24
U16 = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half the smallest subnormal
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def rng(*seed):
    return np.random.default_rng(list(seed))


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


class Cache:
    """A pool with sequences of the given lengths in scattered pages.  Every
    place that no token owns holds `junk` (NaN by default)."""

    def __init__(self, mm, g, lengths, H, D, ps, cache, dtype=None, junk=float("nan"), extra=3,
                 width=None, kscale=1.0):
        self.ps, self.H, self.D, self.lengths = ps, H, D, list(lengths)
        pages = [-(-n // ps) for n in lengths]
        P = sum(pages) + extra
        ids = g.permutation(P)
        width = max(pages + [1]) if width is None else width
        table = np.full((max(len(lengths), 1), width), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = ids[at:at + n]
            at += n
        self.table_np = table
        self.dtype = DTYPES[cache] if cache != "i8" else torch.int8
        i8 = cache == "i8"
        k = np.full((P, H, ps, D), 0 if i8 else junk, np.float32)
        v = np.full((P, H, D, ps), 0 if i8 else junk, np.float32)
        ks = np.full((P, H, ps), junk, np.float32)
        vs = np.full((P, H, ps), junk, np.float32)
        for b, n in enumerate(lengths):
            for t in range(n):
                p, s = table[b, t // ps], t % ps
                if i8:
                    k[p, :, s] = g.integers(-127, 128, (H, D))
                    v[p, :, :, s] = g.integers(-127, 128, (H, D))
                    ks[p, :, s] = kscale * g.uniform(0.5, 3.0, H)
                    vs[p, :, s] = g.uniform(0.5, 3.0, H)
                else:
                    k[p, :, s] = kscale * g.standard_normal((H, D))
                    v[p, :, :, s] = g.standard_normal((H, D))
        self.k, self.v = dev(k, self.dtype), dev(v, self.dtype)
        self.ks, self.vs = (dev(ks), dev(vs)) if i8 else (None, None)
        self.kv = mm.PagedKV(self.k, self.v, self.ks, self.vs)
        self.table = dev(table)
        self.len = torch.tensor(self.lengths or [0], dtype=torch.int32, device="cuda")

    def rows(self, b, h, lo, n):
        """(k, v) float64 [n - lo][D] of sequence b, kv head h."""
        if not hasattr(self, "_values"):  # of the pool as it was made
            k64, v64 = f64(self.k), f64(self.v)
            if self.ks is not None:
                k64 = k64 * (f64(self.ks) / 127)[..., None]
                v64 = v64 * (f64(self.vs) / 127)[:, :, None, :]
            self._values = k64, v64
        k64, v64 = self._values
        K = np.zeros((n - lo, self.D))
        V = np.zeros((n - lo, self.D))
        for t in range(lo, n):
            p, s = self.table_np[b, t // self.ps], t % self.ps
            K[t - lo], V[t - lo] = k64[p, h, s], v64[p, h, :, s]
        return K, V


def attention_reference(ref, c, q, lengths, scale, window, softcap, rows=None):
    """out, lse and their bounds' ingredients for every sequence and head."""
    q64 = f64(q)
    B, Hq, D = q64.shape
    G = Hq // c.H
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    pv, mag = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    for b in range(B):
        r = b if rows is None else rows[b]
        n = lengths[r] if 0 <= r < len(lengths) else 0
        lo = max(0, n - window) if window > 0 else 0
        for h in range(c.H):
            k, v = c.rows(r, h, lo, n) if n > lo else (np.zeros((0, D)), np.zeros((0, D)))
            at = slice(h * G, (h + 1) * G)
            out[b, at], lse[b, at], pv[b, at], mag[b, at] = ref.attention_rows(
                q64[b, at], k, v, scale, softcap)
    return out, lse, pv, mag


def check_attention(got, got_lse, want, want_lse, pv, mag, D, T, softcap=0.0):
    """fp32 scores: each of D products and sums, the scale, the cap and exp2's
    argument round once, so a score is off by at most (D + 8) u32 of
    sum |q||k| |scale| (+ 4 u32 of the cap) and a probability by that much
    relatively, twice over for the maximum; P enters the matrix cores with 16
    bits or more (2^-16); up to T + 8 terms are summed in fp32."""
    ds = (D + 8) * U32 * mag + (8 * U32 * softcap) + 8 * U32 * np.abs(
        np.where(np.isfinite(want_lse), want_lse, 0))
    eps = 2 * ds + 2.0 ** -16 + (T + 16) * U32
    bound = U16[got.dtype] * np.abs(want) + eps[..., None] * pv + TINY[got.dtype]
    d = np.abs(f64(got) - want)
    assert np.array_equal(np.isfinite(f64(got)), np.isfinite(want))
    bad = d > bound * (1 + 2.0 ** -8)
    assert not bad.any(), (np.argwhere(bad)[:4], d[bad][:4], bound[bad][:4])
    l = f64(got_lse)
    empty = ~np.isfinite(want_lse)
    assert np.array_equal(l[empty], want_lse[empty])
    lb = ds + (T + 16) * U32 + 4 * U32 * np.abs(np.where(empty, 0, want_lse))
    dl = np.abs(np.where(empty, 0, l) - np.where(empty, 0, want_lse))
    assert np.all(dl <= lb), (dl.max(), lb[np.unravel_index(dl.argmax(), dl.shape)])
