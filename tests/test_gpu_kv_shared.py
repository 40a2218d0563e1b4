"""kv_attention_shared against the definition in 64 bits (the bounds are
kv_attention's: see serving_cases), and beside kv_attention on the same pages."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import serving_cases as sc
from oracle import serving_ref as ref

pytestmark = pytest.mark.gpu


class Shared:
    """Sequences of the given lengths that begin with the same n0 tokens.  Whole
    pages of the prefix are in no table (entries `hidden`), the rest of each
    sequence is in pages of its own; places that no token owns, a prefix's last
    ones in the sequences' own pages among them, hold `junk`."""

    def __init__(self, mm, g, n0, lengths, H, D, ps, cache, junk=float("nan"), hidden=-1, kscale=1.0):
        self.ps, self.H, self.D, self.n0, self.lengths = ps, H, D, n0, list(lengths)
        i8 = cache == "i8"
        first, whole = -(-n0 // ps), n0 // ps
        mine = [max(0, -(-n // ps) - whole) for n in lengths]
        P = first + sum(mine) + 2
        ids = g.permutation(P)
        width = max([-(-n // ps) for n in lengths] + [1])
        table = np.full((len(lengths), width), hidden, np.int32)
        at = first
        for b, m in enumerate(mine):
            table[b, whole:whole + m] = ids[at:at + m]
            at += m
        self.pages_np, self.table_np = ids[:first].astype(np.int32), table
        k = np.full((P, H, ps, D), 0 if i8 else junk, np.float32)
        v = np.full((P, H, D, ps), 0 if i8 else junk, np.float32)
        ks, vs = np.full((P, H, ps), junk, np.float32), np.full((P, H, ps), junk, np.float32)

        def put(p, s):
            if i8:
                k[p, :, s], v[p, :, :, s] = g.integers(-127, 128, (2, H, D))
                ks[p, :, s], vs[p, :, s] = kscale * g.uniform(0.5, 3.0, H), g.uniform(0.5, 3.0, H)
            else:
                k[p, :, s], v[p, :, :, s] = kscale * g.standard_normal((H, D)), g.standard_normal((H, D))
        for t in range(n0):
            put(ids[t // ps], t % ps)
        for b, n in enumerate(lengths):
            for t in range(n0, n):
                put(table[b, t // ps], t % ps)
        t = torch.int8 if i8 else sc.DTYPES[cache]
        self.k, self.v = sc.dev(k, t), sc.dev(v, t)
        self.ks, self.vs = (sc.dev(ks), sc.dev(vs)) if i8 else (None, None)
        self.kv = mm.PagedKV(self.k, self.v, self.ks, self.vs)
        self.table, self.pages = sc.dev(table), sc.dev(self.pages_np)
        self.len = sc.dev(np.array(lengths, np.int32))

    def place(self, b, t):
        page = self.pages_np[t // self.ps] if t < self.n0 else self.table_np[b, t // self.ps]
        return page, t % self.ps

    def rows(self, b, h, lo, n):
        if not hasattr(self, "_values"):
            k64, v64 = sc.f64(self.k), sc.f64(self.v)
            if self.ks is not None:
                k64 = k64 * (sc.f64(self.ks) / 127)[..., None]
                v64 = v64 * (sc.f64(self.vs) / 127)[:, :, None, :]
            self._values = k64, v64
        k64, v64 = self._values
        at = [self.place(b, t) for t in range(lo, n)]
        p, s = np.array([x[0] for x in at]), np.array([x[1] for x in at])
        return k64[p, h, s], v64[p, h, :, s]

    def full_table(self):
        """The tables as forks leave them, for kv_attention."""
        t = self.table_np.copy()
        t[:, :self.n0 // self.ps] = self.pages_np[:self.n0 // self.ps]
        return sc.dev(t)


def queries(g, B, Hq, D, t):
    return sc.dev(g.standard_normal((B, Hq, D)).astype(np.float32), t)


def check(mm, c, q, window=0, softcap=0.0, scale=None, rows=None, **kw):
    scale = c.D ** -0.5 if scale is None else scale
    out, lse = mm.kv_attention_shared(q, c.kv, c.table, c.len, c.pages, c.n0, rows=rows, scale=scale,
                                      window=window, softcap=softcap, return_lse=True, **kw)
    r = None if rows is None else rows.tolist()
    want = sc.attention_reference(ref, c, q, c.lengths, scale, window, softcap, r)
    sc.check_attention(out, lse, *want, c.D, max(c.lengths + [1]), softcap)
    return out, lse


SIZES = [
    # B, Hq, Hkv, D, page, prefix, longest own
    (1, 1, 1, 64, 16, 1, 1), (1, 4, 4, 128, 16, 100, 5), (2, 8, 2, 128, 16, 333, 40),
    (4, 4, 1, 128, 32, 257, 3), (5, 4, 1, 128, 16, 64, 100), (17, 8, 2, 128, 16, 300, 30),
    (9, 16, 2, 64, 64, 500, 70), (70, 2, 2, 64, 16, 130, 20), (33, 4, 2, 80, 16, 200, 20),
    (20, 6, 2, 96, 32, 150, 33), (12, 6, 2, 192, 16, 190, 20), (10, 4, 2, 256, 16, 170, 17),
    (3, 34, 2, 128, 16, 150, 20), (2, 2, 1, 16, 16, 40, 9), (3, 2, 1, 160, 128, 700, 9),
    (2, 4, 2, 128, 1024, 1500, 300),
]


@pytest.mark.parametrize("cache,dtype", [("f16", "f16"), ("bf16", "bf16"), ("i8", "f16"), ("i8", "bf16")])
@pytest.mark.parametrize("B,Hq,H,D,ps,n0,tail", SIZES)
def test_sizes(lib, B, Hq, H, D, ps, n0, tail, cache, dtype):
    g = sc.rng(1, B, Hq, D, n0)
    lengths = [n0 + int(x) for x in g.integers(0, tail + 1, B)]
    lengths[-1] = n0 + tail
    c = Shared(lib, g, n0, lengths, H, D, ps, cache)
    check(lib, c, queries(g, B, Hq, D, sc.DTYPES[dtype]))


@pytest.mark.parametrize("cache,dtype", [("f16", "f16"), ("bf16", "bf16"), ("i8", "bf16")])
@pytest.mark.parametrize("B,Hq,H,D", [(3, 4, 2, 128), (24, 8, 2, 128), (20, 4, 1, 64)])
def test_short_and_empty_rows(lib, B, Hq, H, D, cache, dtype):
    """Rows shorter than the prefix, of length 0, below 0, and rows that do not
    exist, beside whole ones."""
    g = sc.rng(2, B)
    n0 = 200
    lengths = [0 if x < 0.3 else int(n0 * x) if x < 0.7 else n0 + int(30 * x) for x in g.random(B)]
    lengths[0], lengths[1], lengths[2] = 0, 1, n0 + 30
    c = Shared(lib, g, n0, lengths, H, D, 16, cache)
    q = queries(g, B, Hq, D, sc.DTYPES[dtype])
    out, lse = check(lib, c, q)
    assert not out[0].any() and (lse[0] == -math.inf).all()
    rows = g.permutation(np.r_[np.arange(B - 2), -1, B + 5]).astype(np.int32)
    check(lib, c, q, rows=sc.dev(rows))
    c.len[2] = -5
    c.lengths[2] = 0
    check(lib, c, q)


@pytest.mark.parametrize("cache,dtype", [("f16", "f16"), ("bf16", "bf16"), ("i8", "bf16")])
@pytest.mark.parametrize("B,Hq,H,D,window", [
    (3, 8, 8, 128, 0), (5, 6, 2, 64, 0), (4, 4, 2, 96, 700), (1, 20, 1, 128, 0), (17, 2, 2, 128, 0),
    (2, 32, 4, 80, 300), (3, 2, 2, 256, 0),
])
def test_long_own_tokens(lib, B, Hq, H, D, window, cache, dtype):
    """Own tokens dealt out over workgroups beside a prefix of one tile and of two."""
    g = sc.rng(14, B, Hq, D)
    n0 = 150
    lengths = [n0 + int(x) for x in g.integers(300, 1500, B)]
    if B > 2:
        lengths[1], lengths[2] = 40, 0
    c = Shared(lib, g, n0, lengths, H, D, 16, cache)
    check(lib, c, queries(g, B, Hq, D, sc.DTYPES[dtype]), window=window)


@pytest.mark.parametrize("window", [1, 20, 64, 150, 1000])
@pytest.mark.parametrize("cache,dtype", [("f16", "f16"), ("bf16", "bf16"), ("i8", "f16")])
def test_window_and_softcap(lib, cache, dtype, window):
    g = sc.rng(3, window)
    n0 = 180
    lengths = [n0 + int(x) for x in g.integers(0, 100, 21)] + [5, 0, n0]
    c = Shared(lib, g, n0, lengths, 2, 128, 16, cache, kscale=3.0)
    q = queries(g, 24, 4, 128, sc.DTYPES[dtype])
    check(lib, c, q, window=window)
    check(lib, c, q, window=window, softcap=5.0)
    check(lib, c, q, softcap=2.0, scale=0.5)


@pytest.mark.parametrize("cache,dtype", [("f16", "f16"), ("bf16", "bf16"), ("i8", "bf16")])
def test_long(lib, cache, dtype):
    """Several pieces of the prefix and of the sequences' own tokens."""
    g = sc.rng(4)
    n0 = 3001
    c = Shared(lib, g, n0, [n0 + 700, n0, n0 + 1, n0 + 300, 1500], 1, 64, 16, cache)
    check(lib, c, queries(g, 5, 4, 64, sc.DTYPES[dtype]))
    check(lib, c, queries(g, 5, 4, 64, sc.DTYPES[dtype]), max_len=n0 + 700)


def test_many_rows(lib):
    """Thousands of queries on one kv head: many tiles, one piece."""
    g = sc.rng(13)
    n0, B = 50, 2000
    lengths = [n0 + (b % 3) for b in range(B)]
    lengths[77] = 12
    c = Shared(lib, g, n0, lengths, 1, 16, 16, "f16")
    check(lib, c, queries(g, B, 20, 16, torch.float16))


def test_no_prefix_and_nothing_else(lib):
    g = sc.rng(5)
    c = Shared(lib, g, 0, [30, 0, 300], 2, 64, 16, "f16")
    q = queries(g, 3, 4, 64, torch.float16)
    check(lib, c, q)
    c = Shared(lib, g, 64, [64, 64, 64], 2, 64, 16, "f16", hidden=1 << 30)
    check(lib, c, q)
    # a bound below the prefix cuts it
    out, lse = lib.kv_attention_shared(q, c.kv, c.table, c.len, c.pages, 64, max_len=40, return_lse=True)
    c.lengths = [40, 40, 40]
    want = sc.attention_reference(ref, c, q, c.lengths, 0.125, 0, 0.0)
    sc.check_attention(out, lse, *want, 64, 40)
    out, lse = lib.kv_attention_shared(q, c.kv, c.table, c.len, c.pages, 64, max_len=0, return_lse=True)
    assert not out.any() and (lse == -math.inf).all()
    assert lib.kv_attention_shared(q[:0], c.kv, c.table, c.len, c.pages, 64).shape == (0, 4, 64)


def test_beside_kv_attention(lib):
    """The same pages through both, and the same call twice."""
    g = sc.rng(6)
    n0 = 777
    lengths = [n0 + int(x) for x in g.integers(0, 300, 40)]
    c = Shared(lib, g, n0, lengths, 2, 128, 16, "bf16", junk=0.0)
    # the page that the prefix fills partly, as a fork copies it
    k, v = c.k, c.v
    for b, n in enumerate(lengths):
        if n > n0:
            p, src = int(c.table_np[b, n0 // 16]), int(c.pages_np[-1])
            k[p, :, :n0 % 16], v[p, :, :, :n0 % 16] = k[src, :, :n0 % 16], v[src, :, :, :n0 % 16]
    q = queries(g, 40, 8, 128, torch.bfloat16)
    keep = torch.tensor([n > n0 for n in lengths], device="cuda")
    a, la = lib.kv_attention_shared(q, c.kv, c.table, c.len, c.pages, n0, return_lse=True)
    b, lb = lib.kv_attention(q, c.kv, c.full_table(), c.len, return_lse=True)
    # each is within half a step, 2^-8 |x|, of the exact result and 2^-16 of sums
    # of |p v| (at most about 1 here), so two are within twice that of one another
    d = (a.float() - b.float()).abs()[keep]
    far = d > 2.0 ** -7 * a.float().abs()[keep] + 2.0 ** -14
    assert not bool(far.any()), (d[far], a[keep][far])
    assert bool(((la - lb).abs()[keep] < 1e-4).all())
    a2, la2 = lib.kv_attention_shared(q, c.kv, c.table, c.len, c.pages, n0, return_lse=True)
    assert torch.equal(a, a2) and torch.equal(la, la2)


@pytest.mark.parametrize("cache,dtype", [("f16", "f16"), ("bf16", "bf16"), ("i8", "bf16")])
@pytest.mark.parametrize("B", [4, 40])
def test_not_finite(lib, B, cache, dtype):
    """An infinity or NaN reaches the rows that see its token and no others,
    also where short rows and a window end inside the prefix."""
    g = sc.rng(7, B)
    n0, bad = 150, 100
    lengths = [n0 + 20] * B
    for i in range(0, B, 3):
        lengths[i] = int(g.integers(10, bad))
    c = Shared(lib, g, n0, lengths, 1, 64, 16, cache)
    q = queries(g, B, 4, 64, sc.DTYPES[dtype])
    sees = torch.tensor([n > bad for n in lengths], device="cuda")
    page, slot = c.place(0, bad)
    for window in (0, 100):
        clean = lib.kv_attention_shared(q, c.kv, c.table, c.len, c.pages, n0, window=window)
        for what in ("k", "v"):
            for x in (math.nan, math.inf, -math.inf):
                t = {"k": c.ks, "v": c.vs}[what] if cache == "i8" else {"k": c.k, "v": c.v}[what]
                old = t.clone()
                if cache == "i8":
                    t[page, 0, slot] = x
                elif what == "k":
                    t[page, 0, slot, 7] = x
                else:
                    t[page, 0, 7, slot] = x
                got = lib.kv_attention_shared(q, c.kv, c.table, c.len, c.pages, n0, window=window)
                t.copy_(old)
                assert torch.equal(got[~sees], clean[~sees]), (what, x, window)
                if what == "v" and cache != "i8":
                    assert not got[sees][..., 7].isfinite().any()
                    rest = [d for d in range(64) if d != 7]
                    assert got[sees][..., rest].isfinite().all()
                elif math.isnan(x):
                    assert got[sees].isnan().all()


def test_pages_that_do_not_exist(lib):
    """Tokens in prefix pages out of range are not visible."""
    g = sc.rng(8)
    c = Shared(lib, g, 100, [130, 100, 60], 2, 64, 16, "f16")
    q = queries(g, 3, 4, 64, torch.float16)
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1):
        pages = c.pages.clone()
        pages[2] = bad
        out, lse = lib.kv_attention_shared(q, c.kv, c.table, c.len, pages, 100, return_lse=True)
        whole = c.rows
        hole = [t for t in range(32, 48)]

        def rows(b, h, lo, n):
            k, v = whole(b, h, lo, n)
            keep = [i for i, t in enumerate(range(lo, n)) if t not in hole]
            return k[keep], v[keep]
        c.rows = rows
        want = sc.attention_reference(ref, c, q, c.lengths, 0.125, 0, 0.0)
        c.rows = whole
        sc.check_attention(out, lse, *want, 64, 130)


def test_float16_far_from_the_maximum(lib):
    """A token with nearly all probability and no value, the others 2^-12 of it
    and less: their values are the result."""
    g = sc.rng(9)
    n0 = 120
    c = Shared(lib, g, n0, [n0 + 4] * 20, 1, 64, 16, "f16", kscale=0.0)
    p, s = c.place(0, 50)
    q = queries(g, 20, 2, 64, torch.float16)
    q[..., 0] = 1.0
    c.k[p, 0, s] = 0.0
    c.k[p, 0, s, 0] = 8.0 * 1.0397  # exp(8.3178) = 2^12
    c.v[p, 0, :, s] = 0.0
    check(lib, c, q, scale=1.0)


def test_strides_streams_and_graph(lib):
    g = sc.rng(10)
    n0 = 300
    lengths = [n0 + int(x) for x in g.integers(0, 200, 18)]
    c = Shared(lib, g, n0, lengths, 2, 64, 16, "f16")
    wide = queries(g, 18, 8, 64, torch.float16)
    check(lib, c, wide[:, 2:6])                         # heads of a wider product
    odd = queries(g, 18, 4, 65, torch.float16)[..., 1:]  # copied to whole rows
    check(lib, c, odd)
    q = wide[:, :4].contiguous()
    out = torch.empty_like(q)
    ws = torch.empty(lib.kv_attention_shared_workspace_size(18, 4, 2, 64, n0, n0 + 200),
                     dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        lib.kv_attention_shared(q, c.kv, c.table, c.len, c.pages, n0, max_len=n0 + 200, out=out,
                                workspace=ws)
    for i in range(3):
        q.copy_(queries(g, 18, 4, 64, torch.float16))
        c.len.copy_(torch.tensor([n0 + (7 * i + b) % (n - n0 + 1) for b, n in enumerate(lengths)]))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        want = lib.kv_attention_shared(q, c.kv, c.table, c.len, c.pages, n0, max_len=n0 + 200)
        assert torch.equal(out, want)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = lib.kv_attention_shared(q, c.kv, c.table, c.len, c.pages, n0, max_len=n0 + 200)
    s.synchronize()
    assert torch.equal(a, out)


def test_forked_cache(lib):
    """A prompt forked with PagedKVCache, decoded on and attended together."""
    g = sc.rng(11)
    H, D, n0, B = 2, 64, 45, 6

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def kv(T):
        return [sc.dev(g.standard_normal((T, H, D)).astype(np.float32), torch.float16) for _ in range(2)]
    c = lib.PagedKVCache(100, H, D, page_size=16, max_seqs=B + 1, max_len=100)
    plan = c.extend(i32([0]), i32([n0]), n0)
    c.append(0, *kv(n0), plan.token_rows, plan.positions)
    kids = i32(list(range(1, B + 1)))
    assert c.fork(i32([0] * B), kids).tolist() == [0] * B
    for step in range(20):
        plan = c.extend(kids, i32([1] * B), B)
        c.append(0, *kv(B), plan.token_rows, plan.positions)
        q = queries(g, B, 4, D, torch.float16)
        a, la = c.attend_shared(0, q, 0, n0, rows=kids, return_lse=True)
        b, lb = c.attend(0, q, rows=kids, return_lse=True)
        assert bool(((a.float() - b.float()).abs() <= 2.0 ** -10 * b.float().abs() + 2.0 ** -14).all())
        assert bool(((la - lb).abs() < 1e-4).all())
    c.free(i32([0]))  # any living row knows the prefix's pages
    assert torch.equal(c.attend_shared(0, q, 3, n0, rows=kids), a)


def test_arguments(lib):
    g = sc.rng(12)
    c = Shared(lib, g, 40, [50, 60], 2, 64, 16, "f16")
    q = queries(g, 2, 4, 64, torch.float16)

    def bad(err, *a, **kw):
        with pytest.raises(err):
            lib.kv_attention_shared(*a, **kw)
    bad(ValueError, q, c.kv, c.table, c.len, c.pages, 49)       # three pages hold 48
    bad(ValueError, q, c.kv, c.table, c.len, c.pages, -1)
    bad(TypeError, q, c.kv, c.table, c.len, c.pages.long(), 40)
    bad(ValueError, q, c.kv, c.table, c.len, c.pages.view(1, 3), 40)
    bad(ValueError, q, c.kv, c.table, c.len, c.pages.cpu(), 40)
    bad(TypeError, q.bfloat16(), c.kv, c.table, c.len, c.pages, 40)
    bad(ValueError, q[:, :3], c.kv, c.table, c.len, c.pages, 40)
    bad(ValueError, q[..., :32], c.kv, c.table, c.len, c.pages, 40)
    bad(ValueError, q, c.kv, c.table, c.len[:1], c.pages, 40)
    bad(lib.Int8mmError, q, c.kv, c.table, c.len, c.pages, 40, window=-1)
    bad(lib.Int8mmError, q, c.kv, c.table, c.len, c.pages, 40, scale=math.nan)
    bad(lib.Int8mmError, q, c.kv, c.table, c.len, c.pages, 40,
        workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert lib.kv_attention_shared_workspace_size(2, 3, 2, 64, 40, 100) == 0
