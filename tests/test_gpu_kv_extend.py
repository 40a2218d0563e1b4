"""kv_pages_extend against lists: pages, lengths, statuses and the token maps
are whole numbers and have to be equal."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import serving_cases as sc
from oracle import step_ref as ref

pytestmark = pytest.mark.gpu


def state(g, S, P, ps, width, most):
    """Rows with up to `most` tokens in scattered pages, as far as the pool goes."""
    table, lengths = np.full((S, width), -1, np.int32), np.zeros(S, np.int32)
    count = np.zeros(P, np.int32)
    ids, at = g.permutation(P), 0
    for r in range(S):
        n = int(g.integers(0, most + 1))
        k = -(-n // ps)
        if at + k > P * 2 // 3:
            break
        table[r, :k], lengths[r] = ids[at:at + k], n
        count[ids[at:at + k]] = 1
        at += k
    return table, lengths, count


def both(lib, table, lengths, count, rows, counts, total, ps):
    t, n, c = sc.dev(table), sc.dev(lengths), sc.dev(count)
    plan = lib.kv_pages_extend(t, n, c, sc.dev(np.array(rows, np.int32)),
                               sc.dev(np.array(counts, np.int32)), total, ps)
    lt, ln, lc = table.tolist(), lengths.tolist(), count.tolist()
    want = ref.extend(lt, ln, lc, list(rows), list(counts), total, ps)
    for got, x, name in zip(plan, want, plan._fields):
        assert got.tolist() == x, name
    assert t.tolist() == lt and n.tolist() == ln and c.tolist() == lc
    return plan, (t, n, c)


@pytest.mark.parametrize("S,P,ps,width,n,pad", [
    (1, 8, 16, 8, 1, 0), (5, 40, 16, 6, 3, 7), (64, 900, 16, 20, 64, 0), (64, 5000, 32, 9, 40, 1),
    (300, 13000, 16, 40, 256, 100), (2500, 20000, 16, 12, 1500, 0), (2500, 20000, 16, 12, 2500, 3),
    (40, 30, 64, 8, 33, 5), (1024, 16384, 16, 20, 1024, 9), (1100, 16384, 16, 20, 1025, 0),
    (900, 16385, 16, 20, 300, 0), (400, 16000, 64, 20, 300, 0),
])
def test_extend(lib, S, P, ps, width, n, pad):
    g = sc.rng(1, S, P, n)
    table, lengths, count = state(g, S, P, ps, width, width * ps * 2 // 3)
    rows = g.permutation(S)[:n].tolist()
    counts = [int(x) for x in g.integers(0, width * ps // 3, n)]
    both(lib, table, lengths, count, rows, counts, sum(counts) + pad, ps)
    both(lib, table, lengths, count, rows, [1] * n, n, ps)  # a decode step


# pages in use behind the others: a pool of more than 8192 takes two launches
POOLS = [0, 20000]


@pytest.mark.parametrize("used", POOLS)
def test_refused_requests(lib, used):
    """Rows out of range, named twice, too long, negative counts, a count at
    int32's end, and what follows them."""
    g = sc.rng(2)
    table, lengths, count = state(g, 12, 60, 16, 4, 30)
    count = np.r_[count, np.ones(used, np.int32)]
    lengths[7] = -3  # a row that something else broke
    big = 2 ** 31 - 1
    rows = [3, -1, 12, 3, 4, 5, 6, 7, 4, 8, big, -big - 1, 9, 0]
    counts = [5, 4, 2, 3, 65, -2, 16, 1, 1, 0, 7, 1, 8, 2]
    plan, _ = both(lib, table, lengths, count, rows, counts, 140, 16)
    assert set(plan.status.tolist()) == {0, 2}
    both(lib, table, lengths, count, [1, 2, 3], [5, big, 4], 1000, 16)
    both(lib, table, lengths, count, [1, 2, 3], [big, big, big], 5, 16)
    both(lib, table, lengths, count, [1, 2, 3], [5, 4, 3], 9, 16)    # the third passes total
    both(lib, table, lengths, count, [1, 2, 3], [5, 4, 3], 0, 16)
    both(lib, table, lengths, count, [1, 2], [0, 0], 0, 16)
    both(lib, table, lengths, count, [], [], 0, 16)
    both(lib, table, lengths, count, [], [], 70, 16)


@pytest.mark.parametrize("used", POOLS)
@pytest.mark.parametrize("free", [0, 1, 3, 6])
def test_pages_run_out(lib, free, used):
    """Those that fit in order are done, the others unchanged, their tokens -1."""
    table = np.full((6, 5), -1, np.int32)
    count = np.ones(20, np.int32)
    count[np.arange(free) * 3] = 0
    count = np.r_[count, np.ones(used, np.int32)]
    lengths = np.array([0, 0, 0, 0, 0, 0], np.int32)
    table[5, 0], lengths[5] = 1, 3
    plan, _ = both(lib, table, lengths, count, [0, 1, 5, 2, 3], [20, 33, 13, 16, 0], 82, 16)
    assert plan.status.tolist()[2] == plan.status.tolist()[4] == 0  # need no page
    empty = np.zeros(0, np.int32)
    both(lib, table, np.zeros(6, np.int32), empty, [0, 1], [1, 0], 1, 16)


@pytest.mark.parametrize("P", [4096, 4097, 8192, 8193])
@pytest.mark.parametrize("total", [4096, 4097])
@pytest.mark.parametrize("n", [1, 1024, 1025])
def test_one_launch_or_two(lib, P, total, n):
    """Both sides of what one launch takes, the free pages at the pool's end."""
    count = np.ones(P, np.int32)
    count[P - 700:] = 0
    table, lengths = np.full((n, 300), -1, np.int32), np.zeros(n, np.int32)
    counts = [total // n] * n
    counts[-1] += total - sum(counts)
    both(lib, table, lengths, count, list(range(n)), counts, total, 16)


def test_many_pages(lib):
    g = sc.rng(3)
    P = 300000
    count = (g.random(P) < 0.97).astype(np.int32)
    table, lengths = np.full((70, 40), -1, np.int32), np.zeros(70, np.int32)
    both(lib, table, lengths, count, list(range(70)), [int(x) for x in g.integers(0, 600, 70)],
         70 * 600, 16)


def test_cache_step(lib):
    """A mixed batch, a prompt beside new tokens, written and read back."""
    g = sc.rng(4)
    c = lib.PagedKVCache(64, 2, 32, page_size=16, layers=1, max_seqs=5, max_len=200)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    seen = {}
    for rows, counts in (([0, 2], [20, 1]), ([2, 4, 0], [1, 37, 1]), ([4, 0, 2], [1, 1, 1])):
        plan = c.extend(i32(rows), i32(counts), sum(counts) + 2)
        assert plan.status.tolist() == [0] * len(rows)
        T = sum(counts) + 2
        k, v = [sc.dev(g.standard_normal((T, 2, 32)).astype(np.float32), torch.float16)
                for _ in range(2)]
        c.append(0, k, v, plan.token_rows, plan.positions)
        at = plan.starts.tolist()
        for i, r in enumerate(rows):
            old = seen.get(r, (k[:0], v[:0]))
            seen[r] = tuple(torch.cat((x, y[at[i]:at[i + 1]])) for x, y in zip(old, (k, v)))
    for r, (k, v) in seen.items():
        n = k.shape[0]
        assert int(c.lengths[r]) == n
        a, b = c.gather(0, torch.full((n,), r, dtype=torch.int32, device="cuda"),
                        torch.arange(n, dtype=torch.int32, device="cuda"))
        assert torch.equal(a, k) and torch.equal(b, v)


def test_graph(lib):
    """Captured once, replayed as sequences grow."""
    c = lib.PagedKVCache(100, 1, 16, page_size=16, max_seqs=8, max_len=300)
    rows = torch.tensor([5, 1, 6], dtype=torch.int32, device="cuda")
    counts = torch.tensor([1, 1, 1], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        plan = c.extend(rows, counts, 3 * 40)
    c.lengths.zero_()
    c.table.fill_(-1)
    c.refcount.zero_()
    t, n, r = c.table.tolist(), c.lengths.tolist(), c.refcount.tolist()
    for step in ([1, 1, 1], [40, 1, 0], [1, 17, 33], [16, 16, 16]):
        counts.copy_(torch.tensor(step, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = ref.extend(t, n, r, rows.tolist(), step, 120, 16)
        assert [x.tolist() for x in plan] == list(want)
        assert c.table.tolist() == t and c.lengths.tolist() == n and c.refcount.tolist() == r


def test_arguments(lib):
    c = lib.PagedKVCache(8, 1, 16, max_seqs=2)
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    ok = (c.table, c.lengths, c.refcount, i, i, 4, 16)

    def bad(err, at, x):
        a = list(ok)
        a[at] = x
        with pytest.raises(err):
            lib.kv_pages_extend(*a)
    bad(TypeError, 3, i.long())
    bad(ValueError, 4, i[:1])
    bad(ValueError, 3, i.view(1, 2))
    bad(ValueError, 4, i.cpu())
    bad(ValueError, 1, c.lengths[:1])
    bad(ValueError, 2, c.refcount.view(2, 4))
    bad(ValueError, 5, -1)
    bad(lib.Int8mmError, 5, 1 << 28)
    bad(lib.Int8mmError, 6, 20)
    with pytest.raises(lib.Int8mmError):
        lib.kv_pages_extend(*ok, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
