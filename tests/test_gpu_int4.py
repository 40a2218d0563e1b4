"""int4_linear and its weights against the float64 reference: both row types,
every group size, with and without zero points, one row to several passes of
64, odd sizes, strided and unaligned rows, and what is refused."""

import numpy as np
import pytest
import torch

from oracle import serving_ref as ref
from serving_cases import DTYPES, TINY, U16, U32, dev, f64, rng

pytestmark = pytest.mark.gpu


def _case(g, M, K, N, group, zeros, dtype, big=True):
    ng = -(-K // group)
    x = g.standard_normal((M, K))
    if big and K > 4:
        x[:, g.integers(0, K, max(1, K // 100))] *= 30
    X = dev(x.astype(np.float32), DTYPES[dtype])
    codes = g.integers(0, 16, (N, K)).astype(np.uint8)
    scales = g.uniform(0.001, 0.02, (N, ng)).astype(np.float16)
    z = g.integers(0, 16, (N, ng)).astype(np.uint8) if zeros else None
    return X, codes, scales, z


def _check(Y, X, codes, scales, zeros, group, bias=None):
    x = f64(X)
    w = ref.int4_dequant(codes, scales, zeros, group)
    want = x @ w.T
    K = codes.shape[1]
    # fp32 sums of K exact products x * (q + c) with |q + c| <= 143 (bfloat16
    # rows) or 15, the correction by x's own sum and the group's scale: every
    # operation rounds once, relative to sum |x| s (2 * 143 + ..)
    top = 2 * 143 if X.dtype == torch.bfloat16 else 2 * 15
    s = np.repeat(scales.astype(np.float64), group, 1)[:, :K]
    mag = top * (np.abs(x) @ s.T)
    if bias is not None:
        want = want + f64(bias)
        mag = mag + np.abs(f64(bias))
    bound = U16[X.dtype] * np.abs(want) + (K + 16) * U32 * mag + TINY[X.dtype]
    d = np.abs(f64(Y) - want)
    assert np.all(d <= bound * (1 + 2.0 ** -8)), (d - bound).max()


SHAPES = [
    # M, K, N, group
    (1, 1, 1, 32), (1, 8, 1, 128), (2, 31, 5, 32), (1, 32, 64, 32), (3, 33, 65, 32),
    (1, 127, 16, 64), (4, 128, 17, 64), (5, 129, 130, 128), (1, 1024, 1024, 128),
    (7, 520, 300, 64), (15, 200, 70, 256), (16, 640, 48, 128), (17, 384, 100, 128),
    (31, 260, 33, 32), (32, 1000, 90, 64), (33, 136, 257, 128), (48, 320, 65, 32),
    (64, 264, 40, 384), (65, 192, 50, 64), (130, 256, 31, 128), (1, 2200, 24, 128),
    (2, 4100, 16400, 128), (16, 520, 16390, 32), (9, 2048, 100, 1024),
    # K in parts, many channels, tiles of K that end inside a step
    (20, 5300, 70, 64), (64, 5200, 33, 128), (3, 5251, 40, 32), (40, 140, 25700, 128),
    (18, 250, 16, 32), (64, 383, 130, 64),
    (64, 1100, 25650, 32), (24, 1300, 25630, 64), (48, 1288, 25601, 128), (30, 2600, 70, 32),
    (64, 2304, 100, 128),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,K,N,group", SHAPES)
def test_linear(lib, M, K, N, group, zeros, dtype):
    print(f"case int4 {M}x{K}x{N} group={group} zeros={zeros} {dtype}", flush=True)
    g = rng(M, K, N, group, zeros)
    X, codes, scales, z = _case(g, M, K, N, group, zeros, dtype)
    w = lib.int4_pack_weight(dev(codes), dev(scales), None if z is None else dev(z), group)
    bias = dev(g.standard_normal(N).astype(np.float32), X.dtype) if M % 2 else None
    Y = lib.int4_linear(X, w, bias)
    assert Y.shape == (M, N) and Y.dtype == X.dtype
    _check(Y, X, codes, scales, z, group, bias)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,K,group", [(5, 40, 32), (70, 300, 64), (33, 257, 128), (20, 700, 256)])
def test_pack_and_unpack(lib, N, K, group, zeros):
    g = rng(N, K, group)
    _, codes, scales, z = _case(g, 1, K, N, group, zeros, "f16")
    # bits above the code are not part of it
    w = lib.int4_pack_weight(dev(codes | 0xa0), dev(scales), None if z is None else dev(z | 0x30), group)
    c, s, zz = lib.int4_unpack_weight(w)
    assert np.array_equal(c.cpu().numpy(), codes)
    assert np.array_equal(s.cpu().numpy(), scales)
    assert (zz is None) == (z is None) and (z is None or np.array_equal(zz.cpu().numpy(), z))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("N,K,group", [(3, 5, 32), (40, 200, 64), (65, 513, 128), (7, 1300, 512)])
def test_prepare(lib, N, K, group, symmetric, dtype):
    g = rng(N, K, group, symmetric)
    W = dev((g.standard_normal((N, K)) * 0.05).astype(np.float32), DTYPES[dtype])
    W[0] = 0                       # a scale of zero
    if N > 4:
        W[1] = W[1].abs()          # one sign only
        W[2] = W[2] * 2.0 ** -20   # scales that are subnormal float16, or zero
    w = lib.int4_prepare_weight(W, group, symmetric)
    c, s, z = lib.int4_unpack_weight(w)
    rc, rs, rz = ref.int4_quantize(f64(W), group, symmetric)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(c.cpu().numpy(), rc)
    assert (z is None) == (rz is None) and (rz is None or np.array_equal(z.cpu().numpy(), rz))


def test_large_scale_saturates(lib):
    W = torch.full((2, 64), 3.0e6, dtype=torch.bfloat16, device="cuda")
    c, s, _ = lib.int4_unpack_weight(lib.int4_prepare_weight(W, 64))
    assert torch.all(s == 65504) and torch.all(c == 15)


@pytest.mark.parametrize("M,K", [(3, 256), (20, 200)])
def test_strided_and_unaligned_rows(lib, M, K):
    g = rng(M, K)
    X, codes, scales, z = _case(g, M, K + 24, 50, 64, True, "f16")
    codes, scales, z = codes[:, :K], scales[:, :-(-K // 64)], z[:, :-(-K // 64)]
    codes, scales, z = map(np.ascontiguousarray, (codes, scales, z))
    w = lib.int4_pack_weight(dev(codes), dev(scales), dev(z), 64)
    want = lib.int4_linear(X[:, :K].contiguous(), w)
    assert torch.equal(lib.int4_linear(X[:, :K], w), want)           # aligned, ldx > K
    shifted = torch.empty(M * (K + 24) + 1, dtype=torch.float16, device="cuda")[1:].view(M, K + 24)
    shifted.copy_(X)
    assert torch.equal(lib.int4_linear(shifted[:, :K], w), want)     # 2-byte aligned
    assert torch.equal(lib.int4_linear(X[:, 3:3 + K], w), lib.int4_linear(X[:, 3:3 + K].contiguous(), w))


def test_prepare_more_groups_than_one_launch_has_waves(lib):
    """2^26 groups and some: the weight repeats, and so does what is stored."""
    N, K, small = (1 << 17) + 16, 1 << 14, 32
    W = torch.randn((small, K), device="cuda", generator=torch.Generator("cuda").manual_seed(3)).half()
    want = lib.int4_prepare_weight(W, group_size=32)
    got = lib.int4_prepare_weight(W.repeat((N + small - 1) // small, 1)[:N], group_size=32)
    for a, b in ((got.Wq, want.Wq), (got.params, want.params)):
        b = b.view(2, -1)
        a = a.view(-1, b.shape[1])
        assert a.shape[0] == N // 16
        assert bool((a[0::2] == b[0]).all()) and bool((a[1::2] == b[1]).all())


def test_rows_do_not_depend_on_each_other(lib):
    # a row's result is the same alone, among others, and beside rows of NaN
    g = rng(5)
    X, codes, scales, z = _case(g, 16, 384, 80, 128, True, "bf16")
    w = lib.int4_pack_weight(dev(codes), dev(scales), dev(z), 128)
    Y = lib.int4_linear(X, w)
    X2 = X.clone()
    X2[1:] = float("nan")
    assert torch.equal(lib.int4_linear(X2, w)[0], Y[0])
    assert torch.isnan(lib.int4_linear(X2, w)[1:]).all()


def test_infinite_input_stays_in_its_row(lib):
    X = torch.ones((2, 64), dtype=torch.float16, device="cuda")
    X[1, 5] = float("inf")
    codes = torch.full((3, 64), 9, dtype=torch.uint8, device="cuda")
    w = lib.int4_pack_weight(codes, torch.ones((3, 1), dtype=torch.float16, device="cuda"), None, 64)
    Y = lib.int4_linear(X, w)
    assert torch.all(Y[0] == 64) and torch.all(Y[1] == float("inf"))


def test_graph_and_another_stream(lib):
    g = rng(77)
    for M, K, N in ((1, 512, 300), (20, 5300, 70), (3, 77, 50)):
        X, codes, scales, z = _case(g, M, K, N, 64, True, "f16")
        w = lib.int4_pack_weight(dev(codes), dev(scales), dev(z), 64)
        want = lib.int4_linear(X, w)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = lib.int4_linear(X, w)
        side.synchronize()
        assert torch.equal(got, want)
        Y = torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.int4_linear(X, w, out=Y)
        for k in range(3):
            X.copy_(X.roll(1, 0) * 0.5)
            Y.fill_(9)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(Y, lib.int4_linear(X, w))


def test_empty(lib):
    w = lib.int4_pack_weight(torch.zeros((5, 0), dtype=torch.uint8, device="cuda"),
                             torch.zeros((5, 0), dtype=torch.float16, device="cuda"), None, 128)
    b = torch.arange(5, dtype=torch.float16, device="cuda")
    X = torch.empty((3, 0), dtype=torch.float16, device="cuda")
    assert torch.equal(lib.int4_linear(X, w, b), b.expand(3, 5))
    assert not lib.int4_linear(X, w).any()
    w = lib.int4_pack_weight(torch.zeros((5, 32), dtype=torch.uint8, device="cuda"),
                             torch.zeros((5, 1), dtype=torch.float16, device="cuda"), None, 32)
    assert lib.int4_linear(torch.empty((0, 32), dtype=torch.float16, device="cuda"), w).shape == (0, 5)


def test_refusals(lib):
    codes = torch.zeros((4, 64), dtype=torch.uint8, device="cuda")
    sc = torch.ones((4, 1), dtype=torch.float16, device="cuda")
    with pytest.raises(lib.Int8mmError):
        lib.int4_pack_weight(codes, sc, None, 48)
    with pytest.raises(ValueError):
        lib.int4_pack_weight(codes, sc, None, 32)          # scales of another group
    with pytest.raises(TypeError):
        lib.int4_pack_weight(codes, sc.float(), None, 64)
    w = lib.int4_pack_weight(codes, sc, None, 64)
    with pytest.raises(TypeError):
        lib.int4_linear(torch.zeros((1, 64), device="cuda"), w)
    with pytest.raises(ValueError):
        lib.int4_linear(torch.zeros((1, 32), dtype=torch.float16, device="cuda"), w)
    with pytest.raises(ValueError):
        lib.int4_linear(torch.zeros((64, 2), dtype=torch.float16, device="cuda").t(), w)
    with pytest.raises(TypeError):
        lib.int4_linear(torch.zeros((1, 64), dtype=torch.float16, device="cuda"), w,
                        torch.zeros(4, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        lib.int4_linear(torch.zeros((1, 64), dtype=torch.float16), w)


def test_module(lib):
    torch.manual_seed(0)
    for dtype in (torch.float16, torch.bfloat16):
        lin = torch.nn.Linear(200, 96).to(device="cuda", dtype=dtype)
        m = lib.Int4Linear.from_linear(lin, 64, symmetric=False)
        x = torch.randn(2, 3, 200, device="cuda").to(dtype)
        y = m(x)
        assert y.shape == (2, 3, 96) and y.dtype == dtype
        c, s, z = (t.cpu().numpy() for t in lib.int4_unpack_weight(m.weight4))
        _check(y.view(6, 96), x.view(6, 200), c, s, z, 64, m.bias)
        m2 = lib.Int4Linear.from_linear(torch.nn.Linear(200, 96).to(device="cuda", dtype=dtype), 64,
                                        symmetric=False)
        m2.load_state_dict(m.state_dict())
        assert torch.equal(m2(x), y)
