"""Writing, reading and moving a paged cache: kv_append and kv_gather against
the stored layout and the reference quantizer, the page calls against lists
kept by the reference, and a served conversation through PagedKVCache."""

import math

import numpy as np
import pytest
import torch

from oracle import serving_ref as ref
from serving_cases import DTYPES, Cache, attention_reference, check_attention, dev, f64, rng

pytestmark = pytest.mark.gpu

TYPES = [("f16", "f16"), ("bf16", "bf16"), ("i8", "f16"), ("i8", "bf16")]
INT = dict(dtype=torch.int32, device="cuda")


def _i32(a):
    return torch.tensor(list(a), **INT)


def _pool(lib, P, H, ps, D, cache, layers=None):
    dt = DTYPES.get(cache, torch.int8)
    lead = (P, H) if layers is None else (layers, P, H)
    k = torch.zeros((*lead, ps, D), dtype=dt, device="cuda")
    v = torch.zeros((*lead, D, ps), dtype=dt, device="cuda")
    s = [torch.zeros((*lead, ps), device="cuda") for _ in range(2)] if cache == "i8" else [None] * 2
    return lib.PagedKV(k, v, *s)


def _stored(kv, page, slot):
    """(k, v) float64 [H][D] and scales of one place."""
    k, v = f64(kv.k[page, :, slot]), f64(kv.v[page, :, :, slot])
    if kv.k_scale is None:
        return k, v, None, None
    return k, v, f64(kv.k_scale[page, :, slot]), f64(kv.v_scale[page, :, slot])


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("T,H,D,ps,order", [
    (1, 1, 16, 16, "one"), (3, 2, 64, 16, "decode"), (64, 8, 128, 16, "decode"),
    (33, 2, 80, 32, "decode"), (70, 3, 96, 16, "prompt"), (129, 2, 128, 64, "prompt"),
    (100, 1, 256, 32, "late prompt"), (41, 2, 144, 128, "late prompt"), (31, 2, 48, 16, "mixed"),
])
def test_append_and_gather(lib, T, H, D, ps, order, cache, dtype):
    print(f"case append T={T} H={H} D={D} ps={ps} {order} {cache} {dtype}", flush=True)
    g = rng(T, H, D, ps)
    if order in ("one", "decode"):
        rows, pos = np.arange(T), g.integers(0, 3 * ps, T)
    elif order == "mixed":  # two sequences in turns, some places skipped
        rows, pos = np.arange(T) % 2, np.arange(T) * 2
    else:
        start = 0 if order == "prompt" else 13
        rows, pos = np.zeros(T, int), start + np.arange(T)
    S, width = int(rows.max()) + 1, int(pos.max()) // ps + 1
    P = S * width + 2
    table = g.permutation(P)[: S * width].reshape(S, width).astype(np.int32)
    kv = _pool(lib, P, H, ps, D, cache)
    x = g.standard_normal((T, 2, H, D)).astype(np.float32) * g.choice([0.1, 1, 30], (T, 1, H, 1))
    x[0, :, 0] = 0                                         # a row without a scale
    fused = dev(x, DTYPES[dtype])
    k, v = fused[:, 0], fused[:, 1]
    before = kv.k.clone(), kv.v.clone()
    lib.kv_append(k, v, kv, dev(table), _i32(rows), _i32(pos))
    touched = torch.zeros((P, ps), dtype=torch.bool)
    kn, vn = k.float().cpu().numpy(), v.float().cpu().numpy()
    kc, ka = ref.kv_codes(kn)
    vc, va = ref.kv_codes(vn)
    for i in range(T):
        page, slot = table[rows[i], pos[i] // ps], pos[i] % ps
        touched[page, slot] = True
        sk, sv, sks, svs = _stored(kv, page, slot)
        if cache == "i8":
            assert np.array_equal(sk, kc[i]) and np.array_equal(sv, vc[i])
            assert np.array_equal(sks, ka[i]) and np.array_equal(svs, va[i])
        else:
            assert np.array_equal(sk, kn[i]) and np.array_equal(sv, vn[i])
    rest = ~touched.cuda()
    assert torch.equal(kv.k.transpose(1, 2)[rest], before[0].transpose(1, 2)[rest])
    assert torch.equal(kv.v.permute(0, 3, 1, 2)[rest], before[1].permute(0, 3, 1, 2)[rest])

    gk, gv = lib.kv_gather(kv, dev(table), _i32(rows), _i32(pos), dtype=DTYPES[dtype])
    if cache == "i8":
        f32 = np.float32
        for got, c, a in ((gk, kc, ka), (gv, vc, va)):
            want = c.astype(f32) * (a / f32(127))[..., None]
            assert torch.equal(got.cpu(), torch.from_numpy(want).to(DTYPES[dtype]))
    else:
        assert torch.equal(gk, k) and torch.equal(gv, v)


@pytest.mark.parametrize("cache,dtype", TYPES)
def test_places_out_of_range_are_skipped(lib, cache, dtype):
    g = rng(21)
    P, H, ps, D = 6, 2, 16, 64
    table = np.array([[0, 1], [2, -1], [P, 3]], np.int32)
    rows = [0, 1, 1, 2, 2, -1, 3, 0, 0, 1 << 30]
    pos = [31, 15, 16, 0, 16, 0, 0, 32, -1, 5]
    good = [True, True, False, False, True, False, False, False, False, False]
    kv = _pool(lib, P, H, ps, D, cache)
    x = dev(g.standard_normal((2, len(rows), H, D)).astype(np.float32), DTYPES[dtype])
    lib.kv_append(x[0], x[1], kv, dev(table), _i32(rows), _i32(pos))
    gk, gv = lib.kv_gather(kv, dev(table), _i32(rows), _i32(pos), dtype=DTYPES[dtype])
    for i, ok in enumerate(good):
        assert bool(gk[i].any()) == ok and bool(gv[i].any()) == ok
    assert int((kv.k != 0).any(-1).any(1).sum()) == sum(good)


def test_unaligned_rows(lib):
    g = rng(22)
    kv, kv2 = _pool(lib, 2, 2, 16, 64, "i8"), _pool(lib, 2, 2, 16, 64, "i8")
    table = _i32([0, 1]).view(1, 2)
    x = dev(g.standard_normal((20, 2, 64)).astype(np.float32), torch.float16)
    odd = torch.empty(20 * 2 * 65 + 1, dtype=torch.float16, device="cuda")[1:].view(20, 2, 65)
    odd[..., :64] = x
    rows, pos = torch.zeros(20, **INT), torch.arange(20, **INT)
    lib.kv_append(x, x, kv, table, rows, pos)
    lib.kv_append(odd[..., :64], odd[..., :64], kv2, table, rows, pos)
    assert torch.equal(kv.k, kv2.k) and torch.equal(kv.v, kv2.v)
    # a head stride of 0: every head gets the same row
    one = x[:, :1].expand(20, 2, 64)
    lib.kv_append(one, one, kv, table, rows, pos)
    gk, _ = lib.kv_gather(kv, table, rows, pos)
    assert torch.equal(gk[:, 0], gk[:, 1])


def test_non_finite_rows_read_back_as_nan(lib):
    kv = _pool(lib, 1, 1, 16, 64, "i8")
    x = torch.ones((3, 1, 64), dtype=torch.float16, device="cuda")
    x[1, 0, 5], x[2, 0, 6] = math.nan, math.inf
    rows, pos = torch.zeros(3, **INT), torch.arange(3, **INT)
    lib.kv_append(x, x, kv, _i32([0]).view(1, 1), rows, pos)
    k, v = lib.kv_gather(kv, _i32([0]).view(1, 1), rows, pos)
    for t in (k, v):
        assert torch.equal(t[0], x[0])
        assert torch.isnan(t[1]).any() and torch.isnan(t[2]).any()


# ------------------------------------------------------------------ pages

def _fill(kv, g):
    for t in (kv.k, kv.v, kv.k_scale, kv.v_scale):
        if t is not None:
            t.copy_(torch.from_numpy(g.integers(-127, 128, tuple(t.shape)).astype(np.float32)))


def _tensors(kv):
    return [t for t in (kv.k, kv.v, kv.k_scale, kv.v_scale) if t is not None]


def _after(before, copies):
    """The pool's tensors after the copies, all read before they are written."""
    out = []
    for t in before:
        x = t.clone()
        for a, b in copies:
            x[:, b] = t[:, a]
        out.append(x)
    return out


def _same(lib, kv, want, table, lengths, refcount, pool):
    for got, w in zip(_tensors(kv), want):
        assert torch.equal(got, w)
    assert table.cpu().tolist() == pool.table
    if lengths is not None:
        assert lengths.cpu().tolist() == pool.lengths
    assert refcount.cpu().tolist() == pool.ref


def _world(lib, g, S, P, width, ps, cache, layers=2, H=2, D=32, share=True, lengths=None):
    """A pool with sequences in scattered pages, some sharing their first ones."""
    kv = _pool(lib, P, H, ps, D, cache, layers)
    _fill(kv, g)
    ids = list(g.permutation(P))
    table = np.full((S, width), -1, np.int32)
    n = g.integers(0, width * ps + 1, S) if lengths is None else np.array(lengths)
    for s in range(S):
        want = -(-int(n[s]) // ps)
        if want > len(ids):
            n[s], want = len(ids) * ps, len(ids)
        for j in range(want):
            table[s, j] = ids.pop()
    ref_ = np.zeros(P, np.int32)
    if share:
        for s in range(1, S, 3):
            if n[s] >= ps and n[s - 1] >= ps:
                table[s, 0] = table[s - 1, 0]
    for p in table[table >= 0]:
        ref_[p] += 1
    pool = ref.Pool(table, n, ref_, ps)
    return kv, dev(table), dev(n.astype(np.int32)), dev(ref_), pool


@pytest.mark.parametrize("cache", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("layers,H,D,ps", [(1, 1, 16, 16), (3, 2, 64, 16), (2, 8, 128, 64),
                                           (1, 3, 80, 32)])
def test_copy(lib, layers, H, D, ps, cache):
    g = rng(31, layers, H)
    kv = _pool(lib, 12, H, ps, D, cache, layers)
    _fill(kv, g)
    before = [t.clone() for t in _tensors(kv)]
    src, dst = [0, 3, -1, 5, 12, 0, 9], [7, 2, 1, 12, 4, 11, 9]
    lib.kv_pages_copy(kv, _i32(src), _i32(dst))
    for got, w in zip(_tensors(kv), _after(before, [(0, 7), (3, 2), (0, 11)])):
        assert torch.equal(got, w)
    # the pages of a single layer
    one = kv.layer(layers - 1)
    lib.kv_pages_copy(one, _i32([7]), _i32([5]))
    assert torch.equal(one.k[5], one.k[7]) and torch.equal(one.v[5], one.v[7])
    lib.kv_pages_copy(kv, _i32([]), _i32([]))


@pytest.mark.parametrize("cache", ["f16", "i8"])
@pytest.mark.parametrize("S,P,width,ps", [(5, 40, 6, 16), (40, 300, 9, 32), (3, 9000, 70, 16),
                                          (9, 4096, 300, 16), (64, 8192, 130, 64)])
def test_free_and_fork(lib, S, P, width, ps, cache):
    print(f"case fork S={S} P={P} width={width} ps={ps} {cache}", flush=True)
    g = rng(32, S, P)
    kv, table, lengths, refc, pool = _world(lib, g, S, P, width, ps, cache, layers=1, H=1, D=16)
    before = [t.clone() for t in _tensors(kv)]
    order = list(map(int, g.permutation(S)))
    dead, live = order[: S // 2], order[S // 2:]
    named = dead + [dead[0], -1, S, 1 << 30]              # twice, and out of range
    lib.kv_pages_free(table, lengths, refc, _i32(named))
    pool.free(dead)
    _same(lib, kv, before, table, lengths, refc, pool)
    parents = [live[int(i)] for i in g.integers(0, len(live), len(dead))]
    status = lib.kv_pages_fork(kv, table, lengths, refc, _i32(parents), _i32(dead))
    want, copies = pool.fork(parents, dead)
    assert status.cpu().tolist() == want
    _same(lib, kv, _after(before, copies), table, lengths, refc, pool)


def test_fork_refusals_on_the_device(lib):
    g = rng(33)
    # 4 rows hold 3 of 5 pages; two free pages for three partly filled copies
    kv, table, lengths, refc, pool = _world(lib, g, 12, 5, 3, 16, "f16", share=False,
                                            lengths=[20, 16, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0])
    before = [t.clone() for t in _tensors(kv)]
    parents = [0, 1, 0, 0, 1, 0, 0, 12, -1, 2, 4, 0]
    children = [2, 3, 4, 5, 6, 2, 1, 7, 8, 9, 10, 1 << 30]
    status = lib.kv_pages_fork(kv, table, lengths, refc, _i32(parents), _i32(children))
    want, copies = pool.fork(parents, children)
    assert status.cpu().tolist() == want
    assert 1 in want and 2 in want and 0 in want
    _same(lib, kv, _after(before, copies), table, lengths, refc, pool)


@pytest.mark.parametrize("S,P,width,ps", [(4, 30, 8, 16), (50, 200, 12, 32), (3, 20000, 3000, 16),
                                          (1, 4096, 4096, 16), (2, 4097, 2100, 16)])
def test_reserve(lib, S, P, width, ps):
    print(f"case reserve S={S} P={P} width={width} ps={ps}", flush=True)
    g = rng(34, S, P)
    _, table, lengths, refc, pool = _world(lib, g, S, P, width, ps, "f16", layers=1, H=1, D=16,
                                           lengths=g.integers(0, P * ps // S // 2 + 1, S).clip(0, width * ps))
    rows = [int(r) for r in g.permutation(S)] + [0, S, -3]
    new = [min(width * ps, pool.lengths[r] + int(g.integers(0, 2 * P * ps // S // 3 + 2)))
           if 0 <= r < S else 5 for r in rows]
    new[0] = pool.lengths[rows[0]] if S > 1 else new[0]   # nothing to add
    if S > 2:
        new[1] = width * ps + 1                            # too long
        new[2] = pool.lengths[rows[2]] - 1                 # shorter
    for _ in range(2):
        status = lib.kv_pages_reserve(table, lengths, refc, _i32(rows), _i32(new), ps)
        assert status.cpu().tolist() == pool.reserve(rows, new)
        assert table.cpu().tolist() == pool.table
        assert lengths.cpu().tolist() == pool.lengths and refc.cpu().tolist() == pool.ref
        new = [n + ps + 1 for n in new]


@pytest.mark.parametrize("cache", ["f16", "i8"])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("S,P,width,ps", [(4, 30, 5, 16), (30, 200, 5, 32), (5, 9000, 900, 16),
                                          (6, 4096, 100, 16), (0, 10, 1, 16), (70, 64, 1, 16)])
def test_compact(lib, S, P, width, ps, in_place, cache):
    print(f"case compact S={S} P={P} width={width} ps={ps} {cache}", flush=True)
    g = rng(35, S, P)
    kv, table, lengths, refc, pool = _world(lib, g, max(S, 1), P, width, ps, cache, H=1, D=16,
                                            lengths=[0] if S == 0 else None)
    if S > 2:                                              # ids that are none, an unused page
        table[0, -1], table[1, -1] = P, -7
        pool.table[0][-1], pool.table[1][-1] = P, -7
    before = [t.clone() for t in _tensors(kv)]
    out = None if in_place else (torch.empty_like(table), torch.empty_like(refc))
    old = table.clone(), refc.clone()
    t, r, live = lib.kv_pages_compact(kv, table, refc, out=out)
    n, copies = pool.compact()
    assert int(live) == n
    _same(lib, kv, _after(before, copies), t, None, r, pool)
    if not in_place:
        assert torch.equal(table, old[0]) and torch.equal(refc, old[1])
    # a dense pool stays as it is
    kept = [x.clone() for x in _tensors(kv)]
    t2, r2, live2 = lib.kv_pages_compact(kv, t.clone(), r.clone())
    assert int(live2) == n and torch.equal(t2, t) and torch.equal(r2, r)
    assert all(torch.equal(a, b) for a, b in zip(_tensors(kv), kept))


def test_pool_without_pages(lib):
    k = torch.empty((1, 0, 2, 16, 64), dtype=torch.float16, device="cuda")
    kv = lib.PagedKV(k, torch.empty((1, 0, 2, 64, 16), dtype=torch.float16, device="cuda"))
    table, n, ref = torch.full((2, 3), 5, **INT), torch.zeros(2, **INT), torch.zeros(0, **INT)
    t, r, live = lib.kv_pages_compact(kv, table, ref)
    assert int(live) == 0 and t.tolist() == [[-1] * 3] * 2 and r.numel() == 0
    status = lib.kv_pages_reserve(table, n, ref, _i32([0, 1]), _i32([0, 1]), 16)
    assert status.tolist() == [lib.INT8MM_KV_DONE, lib.INT8MM_KV_NO_PAGES] and n.tolist() == [0, 0]
    assert lib.kv_pages_fork(kv, table, n, ref, _i32([0]), _i32([1])).tolist() == [lib.INT8MM_KV_DONE]
    one = kv.layer(0)
    kk, vv = lib.kv_gather(one, table, _i32([0]), _i32([0]))
    assert not kk.any() and not vv.any()
    lib.kv_append(kk, vv, one, table, _i32([0]), _i32([0]))
    out, lse = lib.kv_attention(torch.ones((2, 4, 64), dtype=torch.float16, device="cuda"), one,
                                table, _i32([5, 0]), return_lse=True)
    assert not out.any() and bool((lse == -math.inf).all())


def test_page_calls_replay_from_a_graph(lib):
    g = rng(36)
    kv, table, lengths, refc, pool = _world(lib, g, 8, 60, 6, 16, "f16")
    parents, children = _i32([0, 1, 0]), _i32([5, 6, 7])
    lib.kv_pages_free(table, lengths, refc, children)
    table0, len0, ref0 = table.clone(), lengths.clone(), refc.clone()
    kv0 = [t.clone() for t in _tensors(kv)]

    def step():
        lib.kv_pages_free(table, lengths, refc, children)
        lib.kv_pages_fork(kv, table, lengths, refc, parents, children)
        lib.kv_pages_compact(kv, table, refc)

    def reset():
        table.copy_(table0)
        lengths.copy_(len0)
        refc.copy_(ref0)
        for t, x in zip(_tensors(kv), kv0):
            t.copy_(x)

    step()
    torch.cuda.synchronize()
    want = table.clone(), lengths.clone(), refc.clone(), [t.clone() for t in _tensors(kv)]
    graph = torch.cuda.CUDAGraph()
    reset()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(table, want[0]) and torch.equal(lengths, want[1])
        assert torch.equal(refc, want[2])
        assert all(torch.equal(a, b) for a, b in zip(_tensors(kv), want[3]))


def test_refusals(lib):
    kv = _pool(lib, 4, 2, 16, 64, "f16")
    table, lengths, refc = torch.full((3, 2), -1, **INT), torch.zeros(3, **INT), torch.zeros(4, **INT)
    x = torch.zeros((2, 2, 64), dtype=torch.float16, device="cuda")
    two = _i32([0, 1])
    with pytest.raises(TypeError):
        lib.kv_append(x.bfloat16(), x.bfloat16(), kv, table, two, two)
    with pytest.raises(ValueError):
        lib.kv_append(x, x, kv, table, two, _i32([0]))
    with pytest.raises(ValueError):
        lib.kv_append(x[..., ::2], x[..., ::2], kv, table, two, two)
    with pytest.raises(ValueError):
        lib.kv_append(x, x, _pool(lib, 4, 2, 16, 64, "f16", 1), table, two, two)
    with pytest.raises(TypeError):
        lib.kv_gather(kv, table, two, two, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        lib.kv_gather(kv, table, two.long(), two)
    with pytest.raises(ValueError):
        lib.kv_pages_copy(kv, two, _i32([1]))
    with pytest.raises(ValueError):
        lib.kv_pages_fork(kv, table, lengths, refc[:3], two, two)
    with pytest.raises(ValueError):
        lib.kv_pages_free(table, lengths[:2], refc, two)
    with pytest.raises(lib.Int8mmError):
        lib.kv_pages_reserve(table, lengths, refc, two, two, 24)
    with pytest.raises(lib.Int8mmError):
        lib.kv_pages_fork(kv, table, lengths, refc, two, two,
                          workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        lib.kv_pages_compact(kv, table, refc, out=(table[:2], refc))


# ------------------------------------------------------- a served conversation

@pytest.mark.parametrize("cache,dtype", TYPES)
def test_served_conversation(lib, cache, dtype):
    """A prompt, a fork after some tokens, both branches going on, the first
    freed and the pool compacted: what is attended to is what was written."""
    g = rng(41)
    H, Hq, D, ps, layers = 2, 6, 64, 16, 2
    dt = DTYPES[dtype]
    c = lib.PagedKVCache(40, H, D, ps, layers, max_seqs=4, max_len=200,
                         dtype=DTYPES.get(cache, torch.int8))
    told = {0: [], 2: []}  # the tokens of each row: k, v of every layer

    def say(row, n):
        x = dev(g.standard_normal((n, 2, layers, H, D)).astype(np.float32), dt)
        at = len(told[row])
        rows = torch.full((n,), row, **INT)
        pos = torch.arange(at, at + n, **INT)
        assert not c.reserve(_i32([row]), _i32([at + n])).any()
        for i in range(layers):
            c.append(i, x[:, 0, i], x[:, 1, i], rows, pos)
        told[row] += [x[t] for t in range(n)]

    def check():
        rows = [r for r in told if told[r]]
        for i in range(layers):
            q = dev(g.standard_normal((len(rows), Hq, D)).astype(np.float32), dt)
            out, lse = c.attend(i, q, _i32(rows), return_lse=True)
            for b, r in enumerate(rows):
                x = torch.stack(told[r]).float().cpu().numpy()[:, :, i]  # [T][2][H][D]
                if cache == "i8":
                    code, a = ref.kv_codes(x)
                    x = code * (a.astype(np.float64) / 127)[..., None]
                x = x.astype(np.float64)
                for h in range(H):
                    at = slice(3 * h, 3 * h + 3)
                    w = ref.attention_rows(f64(q[b, at]), x[:, 0, h], x[:, 1, h], D ** -0.5, 0.0)
                    check_attention(out[b:b + 1, at], lse[b:b + 1, at], *[y[None] for y in w], D, len(x))

    say(0, 37)
    check()
    say(0, 1)
    assert c.fork(_i32([0]), _i32([2])).cpu().tolist() == [0]
    told[2] = list(told[0])
    for _ in range(12):
        say(0, 1)
        say(2, 1)
    check()
    c.free(_i32([0]))
    told[0] = []
    live = c.compact()
    assert int(live) == -(-len(told[2]) // ps)
    assert int(c.table.max()) == int(live) - 1
    check()
    say(0, 20)
    check()
