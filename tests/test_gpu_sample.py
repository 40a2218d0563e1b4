"""sample_tokens against the definition in extended precision.  Tokens have to
be equal; the kernel's weights are rounded at 2^-36 (and z in 64 bits), so a
decision nearer than 2^-33 of its mass to its border is open, and the inputs
(seeded) have none."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import serving_cases as sc
from oracle import step_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
OPEN = 2.0 ** -33


def check(lib, x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, exact_ties=False):
    """x a GPU tensor [B][V]; the others numbers or arrays."""
    B = x.shape[0]

    def arg(v, t):
        return sc.dev(np.asarray(v), t) if isinstance(v, (list, np.ndarray)) else v
    got = lib.sample_tokens(x, sc.dev(np.asarray(u, np.float32)), arg(temperature, torch.float32),
                            arg(top_k, torch.int32), arg(top_p, torch.float32),
                            arg(min_p, torch.float32)).tolist()
    f32 = lambda v, b: float(np.float32(v[b] if isinstance(v, (list, np.ndarray)) else v))
    x64 = sc.f64(x)
    for b in range(B):
        k = int(top_k[b]) if isinstance(top_k, (list, np.ndarray)) else top_k
        want, margin = ref.sample(x64[b], f32(u, b), f32(temperature, b), k, f32(top_p, b),
                                  f32(min_p, b))
        assert margin > OPEN or exact_ties, (b, margin)
        assert got[b] == want, (b, got[b], want, margin)
    return got


def logits(g, B, V, spread, t):
    x = spread * g.standard_normal((B, V))
    hot = g.integers(0, V, (B, min(V, 8)))
    np.put_along_axis(x, hot, np.take_along_axis(x, hot, 1) + spread * 3, 1)
    return sc.dev(x.astype(np.float32), t)


FILTERS = [dict(), dict(top_k=1), dict(top_k=40), dict(top_p=0.9), dict(min_p=0.1),
           dict(top_k=50, top_p=0.95, min_p=0.02), dict(temperature=0.0), dict(top_k=700, top_p=0.5),
           dict(temperature=0.3, top_p=0.99), dict(temperature=3.0, top_k=3000, top_p=0.97)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,V,spread", [(1, 1, 1.0), (3, 2, 1.0), (5, 100, 2.0), (4, 8191, 3.0),
                                        (3, 8192, 0.1), (3, 8193, 2.0), (2, 50021, 2.5),
                                        (2, 131072, 0.02), (3, 40000, 8.0)])
def test_filters(lib, B, V, spread, dtype):
    g = sc.rng(1, B, V)
    x = logits(g, B, V, spread, TYPES[dtype])
    for f in FILTERS:
        check(lib, x, g.random(B).astype(np.float32), **f)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_rows_of_their_own(lib, dtype):
    """Different settings in one call, rows of any distance and alignment."""
    g = sc.rng(2)
    B, V = 40, 20011
    wide = logits(g, B, V + 13, 2.0, TYPES[dtype])
    for lead in (0, 1, 3, 8):
        x = wide[:, lead:lead + V]
        check(lib, x, g.random(B).astype(np.float32),
              temperature=g.choice([0.0, 0.5, 1.0, 1.7, -1.0], B), top_k=g.choice([0, -5, 1, 20, 5000, V, V + 9], B),
              top_p=g.choice([0.0, 0.3, 0.9, 1.0, 2.0, -1.0], B),
              min_p=g.choice([0.0, 0.01, 0.3, 1.0, 1.5, -1.0], B))
    one = wide[:1, :V].expand(6, V)  # one row for all
    check(lib, one, np.linspace(0, 0.999, 6, dtype=np.float32), top_p=0.8)


@pytest.mark.parametrize("V", [4, 1024, 20000, 70000])
def test_ties(lib, V):
    """Equal logits: the lower index first, borders that are hit exactly."""
    x = torch.zeros((1, V), device="cuda")
    for u in (0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24):
        assert check(lib, x, [u], exact_ties=True) == [int(u * V)]
        assert check(lib, x, [u], top_k=V // 2, exact_ties=True) == [int(u * (V // 2))]
        assert check(lib, x, [u], top_p=0.5, exact_ties=True) == [int(u * (V // 2))]
        check(lib, x, [u], min_p=1.0, exact_ties=True)
        check(lib, x, [u], top_k=V - 1, top_p=0.25, exact_ties=True)
    # a step of equal logits above others; few values, many equal (zeros of both signs)
    g = sc.rng(3, V)
    x = g.choice([-1.0, -0.0, 0.0, 0.5, 2.0], (3, V)).astype(np.float32)
    for t in TYPES.values():
        for k in (1, 2, V // 3, V // 2, V - 1):
            check(lib, sc.dev(x, t), g.random(3).astype(np.float32), top_k=k, exact_ties=True)
            check(lib, sc.dev(x, t), g.random(3).astype(np.float32), top_k=k, top_p=0.7)


def test_many_close_logits(lib):
    """One bin holds more tokens than are sorted at once, all different."""
    g = sc.rng(4)
    x = sc.dev((1 + 1e-3 * g.standard_normal((2, 100000))).astype(np.float32))
    for f in (dict(top_k=5), dict(top_k=49999), dict(top_p=0.5), dict(top_k=90000, top_p=0.3),
              dict(min_p=0.9995)):
        check(lib, x, g.random(2).astype(np.float32), **f)


def test_many_logits_beside_a_bin(lib):
    """Bins begin at whole sevenths: next to the few tokens of the one that is cut
    lie many more than are listed, too close to tell apart in 32 bits' bounds."""
    g = sc.rng(9)
    x = np.full((2, 9000), np.nextafter(np.float32(3), np.float32(0)), np.float32)
    x[:, 100:110] = 3 + 0.01 * np.arange(10)
    x[:, 200:205] = 5.0
    for f in (dict(top_k=9), dict(top_k=15), dict(top_p=0.04), dict(top_k=700, top_p=0.5)):
        check(lib, sc.dev(x), g.random(2).astype(np.float32), exact_ties=True, **f)
    x = np.full((1, 9000), -3.0, np.float32)  # and from above, below zero
    x[:, 100:110] = np.nextafter(np.float32(-3), np.float32(-4))
    for k in (8995, 3000, 8990, 8991):
        check(lib, sc.dev(x), [0.7], top_k=k, exact_ties=True)


def test_no_distribution(lib):
    """-1 where there is none, and only there; masked tokens are not drawn."""
    g = sc.rng(5)
    inf, nan = math.inf, math.nan
    x = g.standard_normal((9, 9000)).astype(np.float32)
    x[1, 8999], x[2, 17], x[3], x[4, :-1], x[5, 3] = nan, inf, -inf, -inf, -nan
    x[6, ::2] = -inf
    for t in TYPES.values():
        for f in FILTERS:
            got = check(lib, sc.dev(x, t), g.random(9).astype(np.float32), **f)
            assert [i for i, n in enumerate(got) if n == -1] == [1, 2, 3, 5]
            assert got[4] == 8999 and got[6] % 2
    assert lib.sample_tokens(sc.dev(x), torch.zeros(9, device="cuda"), nan).tolist() == [-1] * 9
    assert lib.sample_tokens(torch.empty((2, 0), device="cuda"), torch.zeros(2, device="cuda")).tolist() == [-1, -1]
    assert lib.sample_tokens(torch.empty((0, 5), device="cuda"), torch.zeros(0, device="cuda")).numel() == 0


def test_borders_of_the_arguments(lib):
    """u outside [0, 1), filters that are NaN, temperatures at both ends, far
    and huge logits."""
    g = sc.rng(6)
    x = sc.dev((3 * g.standard_normal((1, 3000))).astype(np.float32))
    for u in (0.0, -1.0, 1.0, 5.0, math.nan, 1 - 2.0 ** -24):
        check(lib, x, [u])
        check(lib, x, [u], top_p=0.6)
    kept = check(lib, x, [0.3])
    assert lib.sample_tokens(x, sc.dev(np.array([0.3], np.float32)), 1.0, 0, math.nan, math.nan).tolist() == kept
    for t in (1e-30, 1e-4, 1e4, 1e30, math.inf):
        for f in (dict(), dict(top_p=0.4), dict(top_k=7), dict(min_p=0.5)):
            check(lib, x, [0.37], temperature=t, exact_ties=True, **f)
    y = x.clone()
    y[0, 0], y[0, 1], y[0, 2] = -1000.0, 3e38, -3e38
    check(lib, y, [0.0])
    check(lib, y, [0.9], temperature=1e38)
    z = torch.tensor([[-70.0, -63.0, 0.0, -1.0]], device="cuda")
    assert check(lib, z, [0.0]) == [1]  # e^-70 is too far
    assert lib.sample_tokens(z, torch.zeros(1, device="cuda"), top_k=1 << 40).tolist() == [1]


def test_same_alone_as_in_a_batch(lib):
    """A row's token depends on nothing but the row, also when called again."""
    g = sc.rng(7)
    x = logits(g, 70, 30000, 2.0, torch.bfloat16)
    u = sc.dev(g.random(70).astype(np.float32))
    a = lib.sample_tokens(x, u, 0.9, 100, 0.95, 0.01)
    for _ in range(3):
        assert torch.equal(lib.sample_tokens(x, u, 0.9, 100, 0.95, 0.01), a)
    for b in (0, 33, 69):
        assert torch.equal(lib.sample_tokens(x[b:b + 1], u[b:b + 1], 0.9, 100, 0.95, 0.01), a[b:b + 1])


def test_frequencies(lib):
    """Drawn often enough, tokens come as often as they should: 20000 draws,
    each count within 5 standard deviations."""
    x = torch.tensor([[0.0, 1.0, -1.0, 2.0, -math.inf, 0.5]], device="cuda").expand(20000, 6)
    u = torch.rand(20000, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    n = torch.bincount(lib.sample_tokens(x, u, 0.7).long(), minlength=6).cpu().double().numpy()
    p = np.exp(np.array([0.0, 1.0, -1.0, 2.0, -np.inf, 0.5]) / 0.7)
    p /= p.sum()
    assert np.all(np.abs(n - 20000 * p) <= 5 * np.sqrt(20000 * p * (1 - p)))


def test_graph(lib):
    g = sc.rng(8)
    x = logits(g, 5, 20000, 2.0, torch.float16)
    u = sc.dev(g.random(5).astype(np.float32))
    top_p = torch.full((5,), 0.9, device="cuda")
    ws = torch.empty(lib.sample_tokens_workspace_size(5, 20000), dtype=torch.uint8, device="cuda")
    out = torch.empty(5, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        lib.sample_tokens(x, u, 0.8, 0, top_p, out=out, workspace=ws)
    for i in range(4):
        x.copy_(logits(g, 5, 20000, 1.0 + i, torch.float16))
        u.copy_(sc.dev(g.random(5).astype(np.float32)))
        top_p.fill_(0.5 + 0.1 * i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lib.sample_tokens(x, u, 0.8, 0, top_p))


def test_arguments(lib):
    x, u = torch.zeros((3, 10), device="cuda"), torch.zeros(3, device="cuda")

    def bad(err, *a, **kw):
        with pytest.raises(err):
            lib.sample_tokens(*a, **kw)
    bad(TypeError, x.double(), u)
    bad(TypeError, x, u.double())
    bad(ValueError, x[0], u)
    bad(ValueError, x.t(), u)
    bad(ValueError, x, u[:2])
    bad(ValueError, x.cpu(), u)
    bad(TypeError, x, u, top_k=torch.zeros(3, device="cuda"))
    bad(ValueError, x, u, top_p=torch.zeros(2, device="cuda"))
    bad(TypeError, x, u, out=torch.zeros(3, dtype=torch.int64, device="cuda"))
    bad(lib.Int8mmError, x, u, workspace=torch.empty(512, dtype=torch.uint8, device="cuda"))
    bad(ValueError, x, u, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    assert lib.sample_tokens_workspace_size(-1, 5) == 0
