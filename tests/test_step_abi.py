"""Host-only checks of the operators around a decode step's attention (no GPU,
no kernel is launched): bad arguments are refused with the documented
statuses before anything is enqueued, and the references on their own terms."""

import math
import os

import numpy as np
import pytest

from int8_quantized_matmul_col_amd import binding, rope, serving
from oracle import step_ref as ref

FAKE = 0x7F0000000000  # never dereferenced
OK, EINVAL, ESHAPE, EWORKSPACE = (binding.INT8MM_OK, binding.INT8MM_EINVAL, binding.INT8MM_ESHAPE,
                                  binding.INT8MM_EWORKSPACE)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from int8_quantized_matmul_col_amd import build
        build.build()
    return serving._lib()


# -------------------------------------------- queries and keys by position

def _rope(lib, q=FAKE, k=FAKE, dt=0, T=3, Hq=4, Hk=2, D=64, qs=(256, 64), ks=(128, 64), p=FAKE,
          turns=FAKE, rot=64, layout=0, factor=1.0, wq=None, wk=None, eps=1e-6, qo=FAKE + 4096,
          ko=FAKE + 8192, qos=(256, 64), kos=(128, 64)):
    return lib.qk_rope(q, k, dt, T, Hq, Hk, D, *qs, *ks, p, turns, rot, layout, factor, wq, wk,
                       eps, qo, ko, *qos, *kos, None)


def test_rope_refusals(lib):
    for n in ("q", "k", "p", "turns", "qo", "ko"):
        assert _rope(lib, **{n: None}) == EINVAL, n
    for n in ("q", "k", "qo", "ko", "wq", "wk"):
        assert _rope(lib, **{n: FAKE + 1}) == EINVAL, n
    assert _rope(lib, p=FAKE + 2) == EINVAL and _rope(lib, turns=FAKE + 4) == EINVAL
    assert _rope(lib, dt=2) == EINVAL and _rope(lib, layout=2) == EINVAL
    for kw in (dict(D=0), dict(D=258), dict(D=65, rot=64), dict(rot=66), dict(rot=-2), dict(rot=31),
               dict(T=-1), dict(T=(1 << 22) + 1), dict(Hq=-1), dict(Hk=-1), dict(Hq=4097),
               dict(Hk=4097), dict(T=1 << 20, Hq=300)):
        assert _rope(lib, **kw) == ESHAPE, kw
    for bad in (math.nan, math.inf):
        assert _rope(lib, factor=bad) == EINVAL and _rope(lib, wq=FAKE, eps=bad) == EINVAL
    assert _rope(lib, wk=FAKE, eps=0.0) == EINVAL and _rope(lib, wk=FAKE, eps=-1.0) == EINVAL
    # outputs that overlap themselves, or their input with other distances
    assert _rope(lib, qos=(256, 63)) == EINVAL and _rope(lib, qos=(63, 256)) == EINVAL
    assert _rope(lib, qos=(200, 64)) == EINVAL and _rope(lib, kos=(0, 64)) == EINVAL
    assert _rope(lib, qo=FAKE, qos=(512, 64)) == EINVAL
    assert _rope(lib, ko=FAKE, kos=(64, 192)) == EINVAL
    assert _rope(lib, T=0) == OK and _rope(lib, Hq=0, Hk=0) == OK
    assert lib.rope_prepare(None, 4, FAKE, None) == EINVAL
    assert lib.rope_prepare(FAKE + 4, 4, FAKE, None) == EINVAL
    assert lib.rope_prepare(FAKE, 129, FAKE, None) == ESHAPE
    assert lib.rope_prepare(FAKE, -1, FAKE, None) == ESHAPE
    assert lib.rope_prepare(None, 0, None, None) == OK


def test_frequencies():
    f = rope.rotary_frequencies
    assert f(0).numel() == 0 and f(2).tolist() == [1.0]
    plain = f(64, 1e4)
    assert np.allclose(plain, [1e4 ** (-i / 32) for i in range(32)], rtol=1e-15)
    assert np.allclose(f(64, 1e4, "linear", 4.0), plain / 4)
    ntk = f(64, 1e4, "ntk", 4.0)
    assert ntk[0] == 1 and math.isclose(ntk[-1], plain[-1] / 4, rel_tol=1e-12)
    parts = f(64, 1e4, "parts", 8.0, original_len=2048, low=1.0, high=32.0)
    turns = 2048 * plain / (2 * math.pi)
    assert np.allclose(parts[turns >= 32], plain[turns >= 32])
    assert np.allclose(parts[turns <= 1], plain[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((parts > plain / 8) & (parts < plain))[mid].all()
    for bad in (dict(rot_dim=3), dict(rot_dim=258), dict(rot_dim=-2), dict(rot_dim=8, theta=0.0),
                dict(rot_dim=8, factor=math.inf), dict(rot_dim=8, scaling="other"),
                dict(rot_dim=8, scaling="parts")):
        with pytest.raises(ValueError):
            f(**bad)
    with pytest.raises(ValueError):
        rope.rotary(8, layout="pairs")
    with pytest.raises(ValueError):
        rope.rotary(8, inv_freq=[1.0, 2.0])
    with pytest.raises(ValueError):
        rope.rotary(4, inv_freq=[1.0, 2.0 ** 20])
    with pytest.raises(ValueError):
        rope.rotary(4, attention_factor=math.nan)


def test_reference_rope():
    g = np.random.default_rng(1)
    x = g.standard_normal((3, 2, 8))
    inv = [1.0, 0.3]
    for layout in ("half", "interleaved"):
        y, _ = ref.rope(x, [0, 5, 100], inv, layout, 1.0, None, 1e-6)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 4:], x[..., 4:])
        assert np.allclose((y * y).sum(-1), (x * x).sum(-1))
    m, n = (0, 2)
    y, _ = ref.rope(x, [0, 5, 100], inv, "half", 1.0, None, 1e-6)
    z = (x[2, 1, m] + 1j * x[2, 1, n]) * np.exp(1j * 100.0)
    assert np.allclose([z.real, z.imag], [y[2, 1, m], y[2, 1, n]])


# --------------------------------------------- the pages of a batch's tokens

def test_extend_refusals(lib):
    def ext(P=8, ps=16, t=FAKE, tr=2, tw=4, l=FAKE, c=FAKE, r=FAKE, k=FAKE, n=2, total=5, st=FAKE,
            starts=FAKE, tok=FAKE, pos=FAKE, ws=FAKE, nb=1 << 20):
        return lib.kv_pages_extend(P, ps, t, tr, tw, l, c, r, k, n, total, st, starts, tok, pos,
                                   ws, nb, None)
    for kw in (dict(ps=20), dict(ps=8), dict(ps=2048), dict(P=-1), dict(P=(1 << 22) + 1),
               dict(n=-1), dict(n=16385), dict(total=-1), dict(total=(1 << 28) - 31), dict(tr=-1),
               dict(tw=1 << 28)):
        assert ext(**kw) == ESHAPE, kw
    for n in ("t", "l", "c", "r", "k", "st", "starts", "tok", "pos"):
        assert ext(**{n: None}) == EINVAL, n
        assert ext(**{n: FAKE + 2}) == EINVAL, n
    assert ext(ws=None) == EWORKSPACE and ext(ws=FAKE + 64) == EWORKSPACE
    assert ext(nb=100) == EWORKSPACE


def test_reference_extend():
    table, n, c = [[4, -1, -1], [-1] * 3], [10, 0], [0, 0, 0, 0, 1]
    got = ref.extend(table, n, c, [1, 0, 1], [20, 7, 1], 30, 16)
    assert got[0] == [0, 0, 2] and got[1] == [0, 20, 27, 28]
    assert got[2] == [1] * 20 + [0] * 7 + [-1] * 3
    assert got[3] == list(range(20)) + list(range(10, 17)) + [-1] * 3
    assert table == [[4, 2, -1], [0, 1, -1]] and n == [17, 20] and c == [1, 1, 1, 0, 1]


# --------------------------------------------------------- the next tokens

def test_sample_refusals(lib):
    need = lib.sample_tokens_workspace_size(3, 10000)
    assert need >= 3 * 2 * 449 * 8
    for bad in ((-1, 5), (5, -1), (65536, 5), (1, (1 << 20) + 1), (65535, 1 << 20)):
        assert lib.sample_tokens_workspace_size(*bad) == 0, bad

    def sam(x=FAKE, dt=3, B=3, V=10000, u=FAKE, t=None, k=None, p=None, m=None, out=FAKE, ws=FAKE,
            nb=need):
        return lib.sample_tokens(x, dt, B, V, V, u, t, 1.0, k, 0, p, 1.0, m, 0.0, out, ws, nb, None)
    for kw in (dict(B=-1), dict(V=-1), dict(B=65536), dict(V=(1 << 20) + 1), dict(B=65535, V=1 << 20)):
        assert sam(**kw) == ESHAPE, kw
    for n in ("x", "u", "out"):
        assert sam(**{n: None}) == EINVAL, n
    for n in ("x", "u", "t", "k", "p", "m", "out"):
        assert sam(**{n: FAKE + 2}) == EINVAL, n
    assert sam(dt=2) == EINVAL and sam(dt=4) == EINVAL and sam(dt=0, x=FAKE + 1) == EINVAL
    assert sam(ws=None) == EWORKSPACE and sam(ws=FAKE + 128) == EWORKSPACE
    assert sam(nb=need - 1) == EWORKSPACE and sam(B=0) == OK


def test_reference_sample():
    x = np.log([0.1, 0.4, 0.2, 0.3])
    pick = lambda u, **kw: ref.sample(x, u, kw.get("t", 1.0), kw.get("k", 0), kw.get("p", 1.0),
                                      kw.get("m", 0.0))[0]
    assert [pick(u) for u in (0.0, 0.05, 0.11, 0.49, 0.51, 0.71)] == [0, 0, 1, 1, 2, 3]
    assert [pick(u, k=2) for u in (0.0, 0.5, 0.6)] == [1, 1, 3]
    assert [pick(u, p=0.75) for u in (0.0, 0.5, 0.7)] == [1, 2, 3]
    assert [pick(u, p=0.7) for u in (0.0, 0.5, 0.7)] == [1, 1, 3]  # 0.7 lies before the third
    assert [pick(u, m=0.6) for u in (0.0, 0.6)] == [1, 3]
    assert pick(0.9, t=0.0) == 1 and pick(0.9, p=0.0) == 1 and pick(0.9, t=1e-3) == 1
    assert ref.sample([0.0, math.nan], 0.5, 1.0, 0, 1.0, 0.0)[0] == -1


# ------------------------------------------------ attention over a shared prefix

def test_shared_attention_refusals(lib):
    from test_serving_abi import _kv
    need = lib.kv_attention_shared_workspace_size(2, 4, 2, 64, 500, 1600)
    assert need > 2 * 4 * 64 * 4

    def att(q=FAKE, dt=0, B=2, Hq=4, qb=256, qh=64, kv=None, t=FAKE, tr=2, tw=100, n=FAKE, rows=None,
            pages=FAKE, n0=500, top=1600, scale=0.1, window=0, cap=0.0, out=FAKE, lse=None, ws=FAKE,
            nb=need):
        return lib.kv_attention_shared(q, dt, B, Hq, qb, qh, kv or _kv(), t, tr, tw, n, rows, pages, n0,
                                       top, scale, window, cap, out, lse, ws, nb, None)
    for n in ("q", "t", "n", "pages", "out"):
        assert att(**{n: None}) == EINVAL, n
    for n in ("t", "n", "pages", "rows", "lse"):
        assert att(**{n: FAKE + 2}) == EINVAL, n
    assert att(q=FAKE + 8) == EINVAL and att(qb=252) == EINVAL and att(qh=60) == EINVAL
    assert att(dt=1) == EINVAL and att(dt=2) == EINVAL
    assert att(kv=_kv(dtype=3)) == EINVAL and att(kv=_kv(page_size=24)) == ESHAPE
    for kw in (dict(Hq=3), dict(Hq=0), dict(B=-1), dict(B=1 << 22), dict(window=-1), dict(top=-1),
               dict(n0=-1), dict(n0=(1 << 30) + 1), dict(tw=1 << 27), dict(tr=-1)):
        assert att(**kw) == ESHAPE, kw
    for bad in (math.nan, math.inf):
        assert att(scale=bad) == EINVAL and att(cap=bad) == EINVAL
    assert att(cap=-1.0) == EINVAL
    assert att(ws=None) == EWORKSPACE and att(ws=FAKE + 16) == EWORKSPACE
    assert att(nb=need - 1) == EWORKSPACE and att(B=0) == OK
    for bad in ((-1, 4, 2, 64, 5, 5), (2, 3, 2, 64, 5, 5), (2, 4, 2, 8, 5, 5), (2, 4, 2, 64, -1, 5),
                (2, 4, 2, 64, 5, -1), (2, 4, 2, 64, (1 << 30) + 1, 5), (0, 4, 2, 64, 5, 5)):
        assert lib.kv_attention_shared_workspace_size(*bad) == 0, bad


def test_shared_workspace_grows_with_the_bound(lib):
    """What is told for a bound serves every shorter one."""
    g = np.random.default_rng(5)
    size = lib.kv_attention_shared_workspace_size
    for _ in range(3000):
        H = int(g.choice([1, 2, 4, 8, 32]))
        Hq, D = H * int(g.choice([1, 2, 4, 8, 16, 17])), int(g.choice([64, 80, 128, 256]))
        B, n0, top = int(g.integers(1, 200)), int(2 ** g.uniform(0, 17)), int(2 ** g.uniform(0, 18))
        assert size(B, Hq, H, D, n0, int(g.integers(0, top + 1))) <= size(B, Hq, H, D, n0, top)
