"""What callers may pass to the serving operators: views whose distances do not
matter, finite values of any size."""

import numpy as np
import pytest
import torch

from serving_cases import Cache, dev, f64, rng
from test_gpu_int4 import _case, _check
from test_gpu_kv_cache import INT, _i32, _pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,Hq", [(1, 4), (1, 1), (3, 1)])
def test_a_distance_that_is_never_used(lib, B, Hq):
    """A dimension of size one may have any stride (a slice of wider rows), and
    torch calls such a view contiguous."""
    g = rng(71, B, Hq)
    c = Cache(lib, g, [40, 17, 300][:B], 1, 64, 16, "f16")
    q = dev(g.standard_normal((B, Hq, 64)).astype(np.float32), torch.float16)
    want = lib.kv_attention(q, c.kv, c.table, c.len)
    buf = torch.zeros(4096, dtype=torch.float16, device="cuda")
    view = buf.as_strided((B, Hq, 64), (257 if B == 1 else Hq * 64, 257 if Hq == 1 else 64, 1))
    view.copy_(q)
    assert view.is_contiguous() and (view.stride(0) % 8 or view.stride(1) % 8)
    assert torch.equal(lib.kv_attention(view, c.kv, c.table, c.len), want)


def test_large_finite_rows_of_an_int8_cache(lib):
    """127 x passes fp32's range from 2.7e36 on; the code does not.  127 x / a =
    10.5 lies on a tie, and ties send the codes through the division."""
    a, x = 254 * 2.0 ** 120, 21 * 2.0 ** 120
    kv = _pool(lib, 1, 1, 16, 64, "i8")
    row = np.zeros((3, 64))
    row[0, :8] = a, x, a / 3, -a / 5, 1e36, -1e30, 1.0, 0.0
    row[1, :4] = 1, 0.5, -0.25, 0.1           # a row beside it
    row[2, :4] = a, a / 3, -a / 7, a / 2
    k = dev(row.astype(np.float32), torch.bfloat16).view(3, 1, 64)
    rows, pos = torch.zeros(3, **INT), torch.arange(3, **INT)
    lib.kv_append(k, k, kv, _i32([0]).view(1, 1), rows, pos)
    held = f64(k)[:, 0]
    top = np.abs(held).max(-1, keepdims=True)
    want = np.rint(127 * held / top)
    for got, scale in ((kv.k[0, 0, :3], kv.k_scale), (kv.v[0, 0, :, :3].t(), kv.v_scale)):
        assert np.array_equal(f64(got), want)
        assert np.array_equal(f64(scale)[0, 0, :3], top[:, 0])
    out = lib.kv_gather(kv, _i32([0]).view(1, 1), rows, pos, dtype=torch.bfloat16)
    for t in out:
        assert torch.isfinite(t).all()


def test_buffers_that_are_not_the_weight(lib):
    """Nothing is launched with buffers elsewhere, or smaller than the sizes say."""
    codes = torch.zeros((40, 300), dtype=torch.uint8, device="cuda")
    w = lib.int4_pack_weight(codes, torch.ones((40, 5), dtype=torch.float16, device="cuda"), None, 64)
    X = torch.zeros((2, 300), dtype=torch.float16, device="cuda")
    assert not lib.int4_linear(X, w).any()
    small = w.Wq[:1024]
    for bad in (dict(Wq=w.Wq.cpu()), dict(params=w.params.cpu()), dict(Wq=small),
                dict(Wq=small[:1].expand(w.Wq.shape)), dict(params=w.params[:-2]),
                dict(params=w.params[::2]), dict(out_features=4096), dict(group_size=32),
                dict(zeros=True), dict(group_size=64, zeros=True)):
        with pytest.raises(ValueError):
            lib.int4_linear(X, w._replace(**bad))
    with pytest.raises(ValueError):
        lib.int4_linear(torch.zeros((2, 400), dtype=torch.float16, device="cuda"),
                        w._replace(in_features=400))
    for group in (0, -64, 48, 96):
        with pytest.raises((ValueError, lib.Int8mmError)):
            lib.int4_linear(X, w._replace(group_size=group))
    with pytest.raises(TypeError):
        lib.int4_linear(X, w._replace(params=None))


def test_workspaces_that_are_none(lib):
    """A workspace on the host, or one whose elements share memory."""
    n = 1 << 22
    one = torch.zeros(1, dtype=torch.uint8, device="cuda")
    c = Cache(lib, rng(72), [5], 2, 64, 16, "f16")
    q = torch.ones((1, 4, 64), dtype=torch.float16, device="cuda")
    codes = torch.zeros((64, 8192), dtype=torch.uint8, device="cuda")
    w = lib.int4_pack_weight(codes, torch.ones((64, 64), dtype=torch.float16, device="cuda"), None, 128)
    X = torch.zeros((20, 8192), dtype=torch.float16, device="cuda")
    table, lengths = torch.full((3, 2), -1, **INT), torch.zeros(3, **INT)
    kv, ref = _pool(lib, 4, 2, 16, 64, "f16"), torch.zeros(4, **INT)
    a, b = _i32([0]), _i32([1])
    wide = c.table.repeat(1, 5000)
    for ws, error in ((torch.zeros(n, dtype=torch.uint8), ValueError), (one.expand(n), ValueError),
                      (n, TypeError)):
        for call in (lambda: lib.int4_linear(X, w, workspace=ws),
                     lambda: lib.kv_attention(q, c.kv, wide, c.len, workspace=ws),
                     lambda: lib.kv_pages_reserve(table, lengths, ref, a, b, 16, workspace=ws),
                     lambda: lib.kv_pages_fork(kv, table, lengths, ref, a, b, workspace=ws),
                     lambda: lib.kv_pages_compact(kv, table, ref, workspace=ws)):
            with pytest.raises(error):
                call()
    # and one of the right kind is taken
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    assert not lib.int4_linear(X, w, workspace=ws).any()
    assert torch.equal(lib.kv_attention(q, c.kv, wide, c.len, workspace=ws),
                       lib.kv_attention(q, c.kv, wide, c.len))
    assert lib.kv_pages_reserve(table, lengths, ref, a, b, 16, workspace=ws).tolist() == [0]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M", [3, 20])
def test_large_bfloat16_rows_of_a_4_bit_product(lib, M, zeros):
    """The stated range: any bfloat16 number below 2^113."""
    g = rng(73, M)
    for group, K in ((32, 256), (128, 256), (256, 1024)):
        X, codes, scales, z = _case(g, M, K, 70, group, zeros, "bf16")
        top = float(np.float32(2.0 ** 113 * (1 - 2.0 ** -8)))
        X = torch.where(X > 0, top, -top).to(torch.bfloat16)
        X[0] = X[0].abs()
        w = lib.int4_pack_weight(dev(codes), dev(scales), None if z is None else dev(z), group)
        Y = lib.int4_linear(X, w)
        assert torch.isfinite(Y).all() and float(X.abs().max()) < 2.0 ** 113
        _check(Y, X, codes, scales, z, group)
