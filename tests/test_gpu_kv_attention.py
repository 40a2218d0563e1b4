"""kv_attention against the float64 reference: cache and row types, head
layouts, head and page sizes, lengths around every tile's edge, windows,
capped scores, splits; what pages hold outside the visible tokens; indexes
out of range; and what is refused."""

import math

import numpy as np
import pytest
import torch

from oracle import serving_ref as ref
from serving_cases import DTYPES, Cache, attention_reference, check_attention, dev, rng

pytestmark = pytest.mark.gpu

TYPES = [("f16", "f16"), ("bf16", "bf16"), ("i8", "f16"), ("i8", "bf16")]


def _run(lib, g, lengths, Hq, H, D, ps, cache, dtype, window=0, softcap=0.0, scale=None, **kw):
    print(f"case attention {lengths} Hq={Hq} H={H} D={D} ps={ps} {cache} {dtype} "
          f"window={window} cap={softcap}", flush=True)
    c = Cache(lib, g, lengths, H, D, ps, cache)
    B = len(lengths)
    q = dev(g.standard_normal((B, Hq, D)).astype(np.float32), DTYPES[dtype])
    s = D ** -0.5 if scale is None else scale
    out, lse = lib.kv_attention(q, c.kv, c.table, c.len, scale=scale, window=window,
                                softcap=softcap, return_lse=True, **kw)
    want = attention_reference(ref, c, q, lengths, s, window, softcap)
    check_attention(out, lse, *want, D, max(lengths + [1]), softcap)
    return c, q, out, lse


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("ps", [16, 32, 64, 256])
def test_lengths(lib, cache, dtype, ps):
    lengths = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 200, 257, 300]
    _run(lib, rng(1, ps), lengths, 8, 2, 64, ps, cache, dtype)


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 240, 256])
def test_head_dims(lib, cache, dtype, D):
    _run(lib, rng(2, D), [5, 70, 131], 6, 2, D, 16, cache, dtype)


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("Hq,H", [(1, 1), (3, 3), (2, 1), (5, 1), (7, 1), (8, 1), (15, 1), (16, 1),
                                  (17, 1), (40, 1), (35, 5), (32, 8)])
def test_head_layouts(lib, cache, dtype, Hq, H):
    _run(lib, rng(3, Hq, H), [0, 37, 90], Hq, H, 128, 32, cache, dtype)


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("window", [1, 2, 16, 17, 63, 64, 65, 100, 299, 300, 1000])
def test_windows(lib, cache, dtype, window):
    _run(lib, rng(4, window), [0, 1, 64, 101, 300], 4, 2, 64, 16, cache, dtype, window=window)


@pytest.mark.parametrize("cache,dtype", TYPES)
def test_softcap(lib, cache, dtype):
    _run(lib, rng(5), [1, 77, 150], 4, 2, 64, 16, cache, dtype, softcap=5.0, scale=0.5)
    _run(lib, rng(5), [1, 77, 150], 4, 2, 64, 16, cache, dtype, softcap=30.0, window=50)


@pytest.mark.parametrize("cache,dtype", TYPES)
def test_steep_scores(lib, cache, dtype):
    # scores of some hundreds: the running maximum moves often, most
    # probabilities vanish
    _run(lib, rng(6), [40, 500, 333], 4, 2, 64, 16, cache, dtype, scale=10.0)
    _run(lib, rng(6), [500], 4, 2, 64, 16, cache, dtype, scale=-2.0)
    _run(lib, rng(6), [500], 4, 2, 64, 16, cache, dtype, scale=0.0)


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("n,ps", [(2049, 16), (5000, 64), (4096, 1024)])
def test_split_lengths(lib, cache, dtype, n, ps):
    _run(lib, rng(7, n), [n], 4, 1, 64, ps, cache, dtype)
    _run(lib, rng(7, n), [n, 3, 0, n // 2], 2, 1, 128, ps, cache, dtype)
    _run(lib, rng(7, n), [n, 900], 2, 1, 64, ps, cache, dtype, window=n // 3)


def test_splits_agree(lib):
    # the bound that the host states changes the split, not the result
    g = rng(8)
    c, q, out, lse = _run(lib, g, [700, 5, 0, 2000], 8, 2, 128, 16, "bf16", "bf16")
    o2, l2 = lib.kv_attention(q, c.kv, c.table, c.len, max_len=2000, return_lse=True)
    wide = torch.full((4, 20000), -1, dtype=torch.int32, device="cuda")
    wide[:, : c.table.shape[1]] = c.table
    o3, l3 = lib.kv_attention(q, c.kv, wide, c.len, return_lse=True)
    for o, l in ((o2, l2), (o3, l3)):
        assert torch.allclose(o.float(), out.float(), rtol=2.0 ** -7, atol=1e-5)
        assert torch.allclose(l, lse, rtol=1e-6, atol=1e-5)
    again = lib.kv_attention(q, c.kv, wide, c.len)
    assert torch.equal(again, o3)


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -65504.0])
def test_what_pages_hold_elsewhere_does_not_matter(lib, cache, dtype, junk):
    lengths = [1, 19, 130, 0, 65]
    res = []
    for j in (0.0, junk):
        g = rng(9)
        c = Cache(lib, g, lengths, 2, 80, 16, cache, junk=j)
        q = dev(g.standard_normal((5, 4, 80)).astype(np.float32), DTYPES[dtype])
        res.append(lib.kv_attention(q, c.kv, c.table, c.len, return_lse=True, window=60))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


def test_before_the_window_pages_may_be_gone(lib):
    g = rng(10)
    c, q, out, _ = _run(lib, g, [400, 333], 4, 2, 64, 16, "f16", "f16", window=100)
    table = c.table.clone()
    table[0, : (400 - 100) // 16] = -1
    table[1, : (333 - 100) // 16] = 1 << 30
    assert torch.equal(lib.kv_attention(q, c.kv, table, c.len, window=100), out)


@pytest.mark.parametrize("cache,dtype", TYPES)
def test_pages_out_of_range_are_not_visible(lib, cache, dtype):
    g = rng(11)
    n, H, D = 150, 2, 64
    c = Cache(lib, g, [n], H, D, 16, cache)
    q = dev(g.standard_normal((1, 4, D)).astype(np.float32), DTYPES[dtype])
    gone = [0, 4, 9]
    bad = c.table.clone()
    bad[0, gone] = torch.tensor([-1, c.k.shape[0], -(1 << 31)], dtype=torch.int32, device="cuda")
    out, lse = lib.kv_attention(q, c.kv, bad, c.len, return_lse=True)
    seen = np.array([t // 16 not in gone for t in range(n)])
    want, wl = np.zeros((1, 4, D)), np.zeros((1, 4))
    pv, mag = np.zeros((1, 4, D)), np.zeros((1, 4))
    q64 = q.cpu().double().numpy()
    for h in range(H):
        k, v = c.rows(0, h, 0, n)
        at = slice(2 * h, 2 * h + 2)
        want[0, at], wl[0, at], pv[0, at], mag[0, at] = ref.attention_rows(
            q64[0, at], k[seen], v[seen], D ** -0.5, 0.0)
    check_attention(out, lse, want, wl, pv, mag, D, n)
    bad[:] = -1
    out, lse = lib.kv_attention(q, c.kv, bad, c.len, return_lse=True)
    assert not out.any() and torch.all(lse == -math.inf)


def test_infinite_and_nan_tokens(lib):
    g = rng(12)
    c = Cache(lib, g, [100, 100, 100], 1, 64, 16, "bf16")
    q = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    q[:, 1] = -1
    t = c.table_np
    c.k[t[0, 2], 0, 3] = -math.inf       # scores -inf for head 0, +inf for head 1
    c.v[t[1, 2], 0, 5, 3] = math.inf     # one value
    c.k[t[2, :7]] = -math.inf            # every score -inf for head 0
    out, lse = lib.kv_attention(q, c.kv, c.table, c.len, return_lse=True)
    assert torch.isfinite(out[0, 0]).all() and torch.isfinite(lse[0, 0])
    assert torch.isnan(out[0, 1]).all()
    assert torch.all(out[1, :, 5] == math.inf)
    assert torch.isfinite(out[1, :, :5]).all() and torch.isfinite(out[1, :, 6:]).all()
    assert not out[2, 0].any() and lse[2, 0] == -math.inf
    c.v[t[1, 2], 0, 5, 3] = math.nan
    out = lib.kv_attention(q, c.kv, c.table, c.len)
    assert torch.isnan(out[1, :, 5]).all() and torch.isfinite(out[1, :, 6:]).all()


def test_rows_lengths_and_bounds(lib):
    g = rng(13)
    lengths = [33, 80, 0, 150]
    c = Cache(lib, g, lengths, 2, 64, 16, "f16")
    rows = [3, 1, 1, -1, 4, 2, 1 << 30]
    q = dev(g.standard_normal((7, 4, 64)).astype(np.float32), torch.float16)
    out, lse = lib.kv_attention(q, c.kv, c.table, c.len, rows=dev(np.array(rows, np.int32)),
                                return_lse=True)
    want = attention_reference(ref, c, q, lengths, 64 ** -0.5, 0, 0.0, rows)
    check_attention(out, lse, *want, 64, 150)
    assert not out[3:].any() and torch.all(lse[3:] == -math.inf)
    # lengths beyond the table or the stated bound are cut, negative ones empty
    far = c.len.clone()
    far[3], far[0], far[1] = 1 << 30, -5, 80
    out = lib.kv_attention(q[:4], c.kv, c.table, far)
    full = c.len.clone()
    full[3], full[0] = c.table.shape[1] * 16, 0
    want = lib.kv_attention(q[:4], c.kv, c.table, full)  # the last page's junk included
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    cut = c.len.clamp(max=70)
    assert torch.equal(lib.kv_attention(q[:4], c.kv, c.table, c.len, max_len=70),
                       lib.kv_attention(q[:4], c.kv, c.table, cut, max_len=70))


def test_strided_queries_and_cache(lib):
    g = rng(14)
    c, q, out, _ = _run(lib, g, [90, 41], 4, 2, 64, 16, "f16", "f16")
    fused = torch.empty((2, 12, 64), dtype=torch.float16, device="cuda")
    fused[:, 3:7] = q
    assert torch.equal(lib.kv_attention(fused[:, 3:7], c.kv, c.table, c.len), out)
    odd = torch.empty(2 * 4 * 65 + 1, dtype=torch.float16, device="cuda")[1:].view(2, 4, 65)
    odd[..., :64] = q
    assert torch.equal(lib.kv_attention(odd[..., :64], c.kv, c.table, c.len), out)
    # a layer of a [pages][layers] pool: pages are not next to each other
    P = c.k.shape[0]
    k = torch.full((P, 3, 2, 16, 64), math.nan, dtype=torch.float16, device="cuda")
    v = torch.full((P, 3, 2, 64, 16), math.nan, dtype=torch.float16, device="cuda")
    k[:, 1], v[:, 1] = c.k, c.v
    kv = lib.PagedKV(k[:, 1], v[:, 1])
    assert torch.equal(lib.kv_attention(q, kv, c.table, c.len), out)


@pytest.mark.parametrize("cache", ["f16", "i8"])
def test_offsets_past_32_bits(lib, cache):
    # pages whose bytes and elements lie beyond 2^32 and 2^31
    H, D, ps = 8, 128, 64
    item = 1 if cache == "i8" else 2
    P = (1 << 32) // (H * ps * D * item) + 40
    g = rng(15)
    small = Cache(lib, g, [300], H, D, ps, cache, extra=0)
    n = small.k.shape[0]
    k = torch.empty((P, H, ps, D), dtype=small.dtype, device="cuda")
    v = torch.empty((P, H, D, ps), dtype=small.dtype, device="cuda")
    ids = torch.arange(P - n, P, device="cuda")
    k[ids], v[ids] = small.k, small.v
    ks = vs = None
    if cache == "i8":
        ks = torch.empty((P, H, ps), device="cuda")
        vs = torch.empty((P, H, ps), device="cuda")
        ks[ids], vs[ids] = small.ks, small.vs
    q = dev(g.standard_normal((1, 16, D)).astype(np.float32), torch.float16)
    want = lib.kv_attention(q, small.kv, small.table, small.len)
    kv = lib.PagedKV(k, v, ks, vs)
    table = small.table + (P - n)
    assert torch.equal(lib.kv_attention(q, kv, table, small.len), want)
    rows = torch.zeros(300, dtype=torch.int32, device="cuda")
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    for a, b in zip(lib.kv_gather(kv, table, rows, pos), lib.kv_gather(small.kv, small.table, rows, pos)):
        assert torch.equal(a, b)


def test_empty_calls(lib):
    c = Cache(lib, rng(16), [5], 2, 64, 16, "f16")
    q = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
    assert lib.kv_attention(q, c.kv, c.table, c.len).shape == (0, 4, 64)
    q = torch.ones((1, 4, 64), dtype=torch.float16, device="cuda")
    none = torch.empty((1, 0), dtype=torch.int32, device="cuda")
    assert not lib.kv_attention(q, c.kv, none, c.len).any()
    kv = lib.PagedKV(c.k[:0], c.v[:0])
    assert not lib.kv_attention(q, kv, c.table, c.len).any()


def test_another_stream_and_graph(lib):
    g = rng(17)
    c, q, out, _ = _run(lib, g, [700, 50], 8, 2, 64, 16, "f16", "f16", max_len=5000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o = lib.kv_attention(q, c.kv, c.table, c.len)
    side.synchronize()
    assert torch.equal(o, out)
    buf = torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.kv_attention(q, c.kv, c.table, c.len, out=buf)
    for n in ([700, 50], [0, 49], [300, 1], [700, 50]):
        c.len.copy_(torch.tensor(n, dtype=torch.int32))
        buf.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, lib.kv_attention(q, c.kv, c.table, c.len))


def test_refusals(lib):
    c = Cache(lib, rng(18), [5], 2, 64, 16, "f16")
    q = torch.ones((1, 4, 64), dtype=torch.float16, device="cuda")
    ok = dict(kv=c.kv, table=c.table, lengths=c.len)
    with pytest.raises(TypeError):
        lib.kv_attention(q.bfloat16(), **ok)
    with pytest.raises(TypeError):
        lib.kv_attention(q.float(), **ok)
    with pytest.raises(ValueError):
        lib.kv_attention(q[:, :3], **ok)                     # 3 heads over 2
    with pytest.raises(ValueError):
        lib.kv_attention(q[..., :32], **ok)
    with pytest.raises(ValueError):
        lib.kv_attention(q.expand(2, 4, 64), **ok)           # more queries than rows
    with pytest.raises(TypeError):
        lib.kv_attention(q, c.kv, c.table.long(), c.len)
    with pytest.raises(ValueError):
        lib.kv_attention(q, c.kv, c.table, c.len.expand(2))
    with pytest.raises(lib.Int8mmError):
        lib.kv_attention(q, softcap=-1.0, **ok)
    with pytest.raises(lib.Int8mmError):
        lib.kv_attention(q, scale=math.inf, **ok)
    with pytest.raises(lib.Int8mmError):
        lib.kv_attention(q, window=-1, **ok)
    with pytest.raises(lib.Int8mmError):
        small = torch.empty(16, dtype=torch.uint8, device="cuda")
        wide = c.table.expand(1, 1).repeat(1, 5000)
        lib.kv_attention(q, c.kv, wide, c.len, workspace=small)
    for k, v in (((4, 2, 24, 64), (4, 2, 64, 24)), ((4, 2, 8, 64), (4, 2, 64, 8)),
                 ((4, 2, 16, 72), (4, 2, 72, 16)), ((4, 2, 16, 272), (4, 2, 272, 16))):
        kv = lib.PagedKV(torch.empty(k, dtype=torch.float16, device="cuda"),
                         torch.empty(v, dtype=torch.float16, device="cuda"))
        with pytest.raises(lib.Int8mmError):
            lib.kv_attention(torch.ones((1, 4, k[3]), dtype=torch.float16, device="cuda"), kv,
                             c.table, c.len)
    with pytest.raises(ValueError):
        lib.PagedKV(c.k, c.k)
    with pytest.raises(ValueError):
        lib.PagedKV(c.k.to(torch.int8), c.v.to(torch.int8))
    with pytest.raises(ValueError):
        lib.PagedKV(c.k.transpose(2, 3), c.v.transpose(2, 3))
    with pytest.raises(TypeError):
        lib.PagedKV(c.k.float(), c.v.float())
    with pytest.raises(ValueError):
        lib.PagedKV(c.k.cpu(), c.v)
