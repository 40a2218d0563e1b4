"""The sizes that a decode step meets and small cases do not reach: many output
channels (several channel tiles a workgroup), many sequences (more than a
wave's lanes hold), rows beside other rows, pages of several slices."""

import numpy as np
import pytest
import torch

from oracle import serving_ref as ref
from serving_cases import DTYPES, Cache, attention_reference, check_attention, dev, f64, rng
from test_gpu_int4 import _case, _check
from test_gpu_kv_cache import _after, _i32, _same, _tensors, _world

pytestmark = pytest.mark.gpu

TYPES = [("f16", "f16"), ("bf16", "bf16"), ("i8", "f16"), ("i8", "bf16")]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("N", [5000, 11008, 13811, 18000, 22000, 28672])
def test_few_rows_of_many_channels(lib, N, dtype):
    g = rng(61, N)
    for group, K in ((32, 264), (64, 392), (128, 1160)):
        for zeros in (False, True):
            X, codes, scales, z = _case(g, 16, K, N, group, zeros, dtype)
            w = lib.int4_pack_weight(dev(codes), dev(scales), None if z is None else dev(z), group)
            bias = dev(g.standard_normal(N).astype(np.float32), X.dtype)
            print(f"case int4 16 and 1x{K}x{N} group={group} zeros={zeros} {dtype}", flush=True)
            Y = lib.int4_linear(X, w, bias)
            _check(Y, X, codes, scales, z, group, bias)
            # a row's sums are the same alone (rows of one launch are independent)
            assert torch.equal(lib.int4_linear(X[5:6], w, bias), Y[5:6])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N,group", [
    (130, 300, 12900, 64), (70, 257, 9000, 32),     # two channel tiles a wave
    (130, 8192, 64, 128), (97, 4100, 130, 64),      # K in parts
])
def test_more_than_64_rows(lib, M, K, N, group, dtype):
    print(f"case int4 {M}x{K}x{N} group={group} {dtype}", flush=True)
    g = rng(62, M, K)
    X, codes, scales, z = _case(g, M, K, N, group, True, dtype)
    w = lib.int4_pack_weight(dev(codes), dev(scales), dev(z), group)
    bias = dev(g.standard_normal(N).astype(np.float32), X.dtype)
    _check(lib.int4_linear(X, w, bias), X, codes, scales, z, group, bias)


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("B", [65, 128, 200])
def test_many_sequences(lib, B, cache, dtype):
    print(f"case attention B={B} {cache} {dtype}", flush=True)
    g = rng(63, B)
    lengths = [int(n) for n in g.integers(257, 600, B)]
    for b in (0, 1, 63, 64, B - 1):  # empty ones, also where a wave's lanes end
        lengths[b] = 0
    for b in (5, B // 2):
        lengths[b] = 1
    c = Cache(lib, g, lengths, 1, 64, 32, cache)
    q = dev(g.standard_normal((B, 2, 64)).astype(np.float32), DTYPES[dtype])
    out, lse = lib.kv_attention(q, c.kv, c.table, c.len, return_lse=True)
    want = attention_reference(ref, c, q, lengths, 64 ** -0.5, 0, 0.0)
    check_attention(out, lse, *want, 64, max(lengths))
    # nearly all of them empty
    few = c.len.clone()
    few[torch.arange(B, device="cuda") != B - 2] = 0
    out, lse = lib.kv_attention(q, c.kv, c.table, few, return_lse=True)
    n = [0] * B
    n[B - 2] = lengths[B - 2]
    want = attention_reference(ref, c, q, n, 64 ** -0.5, 0, 0.0)
    check_attention(out, lse, *want, 64, max(n))


@pytest.mark.parametrize("cache,dtype", TYPES)
def test_a_sequence_beside_others(lib, cache, dtype):
    """The same sequence alone and beside others.  The cuts go by all lengths of
    a call, so other lengths may round differently, within the bound; what the
    others hold does not matter at all."""
    g = rng(64)
    lengths = [700, 400, 0, 2500]
    c = Cache(lib, g, lengths, 2, 64, 16, cache)
    q = dev(g.standard_normal((4, 4, 64)).astype(np.float32), DTYPES[dtype])
    one = attention_reference(ref, c, q[:1], lengths[:1], 64 ** -0.5, 0, 0.0)
    top = max(lengths)

    def attend(n, rows=4, **kw):
        return lib.kv_attention(q[:rows], c.kv, c.table, _i32(n), return_lse=True, max_len=top, **kw)

    first = attend(lengths)
    for n in (lengths, [700, 0, 0, 0], [700, 1, 0, 1], [700, 400, 0, 1234], [700, 399, 0, 2500]):
        out, lse = attend(n)
        check_attention(out[:1], lse[:1], *one, 64, 700)
    out, lse = attend(lengths, rows=1)
    check_attention(out, lse, *one, 64, 700)
    pages = c.table[1:].flatten()
    pages = pages[pages >= 0].long()
    for t in (c.k, c.v):
        t[pages] = t[pages].flip(0)
    out, lse = attend(lengths)
    assert torch.equal(out[0], first[0][0]) and torch.equal(lse[0], first[1][0])
    # up to 256 tokens nothing is cut, and the bits are the same beside any others
    rows = _i32([2, 0, 3])
    short = [lib.kv_attention(q[:3], c.kv, c.table, _i32(n), rows=rows, max_len=256)
             for n in ([200, 0, 150, 0], [256, 0, 150, 7])]
    assert torch.equal(short[0][0], short[1][0])


PAGES = [  # pages of several slices, whole and ragged
    (4, 128, 64, "f16"), (5, 80, 64, "bf16"), (8, 128, 64, "i8"), (3, 176, 128, "i8"),
]


@pytest.mark.parametrize("H,D,ps,cache", PAGES)
def test_fork_of_large_pages(lib, H, D, ps, cache):
    print(f"case fork H={H} D={D} ps={ps} {cache}", flush=True)
    g = rng(65, H, D)
    kv, table, lengths, refc, pool = _world(lib, g, 8, 50, 6, ps, cache, layers=3, H=H, D=D)
    before = [t.clone() for t in _tensors(kv)]
    dead = [6, 1, 3, 4]
    assert any(int(n) for n in lengths[dead])  # rows that hold pages
    lib.kv_pages_free(table, lengths, refc, _i32(dead))
    pool.free(dead)
    parents = [0, 2, 5, 0]
    status = lib.kv_pages_fork(kv, table, lengths, refc, _i32(parents), _i32(dead))
    want, copies = pool.fork(parents, dead)
    assert status.cpu().tolist() == want and copies
    _same(lib, kv, _after(before, copies), table, lengths, refc, pool)


@pytest.mark.parametrize("H,D,ps,cache", PAGES)
def test_compact_of_large_pages(lib, H, D, ps, cache):
    print(f"case compact H={H} D={D} ps={ps} {cache}", flush=True)
    g = rng(66, H, D)
    kv, table, lengths, refc, pool = _world(lib, g, 7, 60, 6, ps, cache, layers=2, H=H, D=D)
    before = [t.clone() for t in _tensors(kv)]
    t, r, live = lib.kv_pages_compact(kv, table, refc)
    n, copies = pool.compact()
    assert int(live) == n and copies
    _same(lib, kv, _after(before, copies), t, None, r, pool)
