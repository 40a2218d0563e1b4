"""Host-only checks of the serving ABI (no GPU, no kernel is launched): the
header, the library's exports and the binding agree, and bad arguments are
refused with the documented statuses before anything is enqueued."""

import ctypes
import math
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

from int8_quantized_matmul_col_amd import binding, serving
from oracle import serving_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "int8mm_serving.h")
FAKE = 0x7F0000000000  # never dereferenced
OK, EINVAL, ESHAPE, EWORKSPACE = (binding.INT8MM_OK, binding.INT8MM_EINVAL, binding.INT8MM_ESHAPE,
                                  binding.INT8MM_EWORKSPACE)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from int8_quantized_matmul_col_amd import build
        build.build()
    return serving._lib()


def _kv(**kw):
    H, ps, D, P = kw.get("kv_heads", 2), kw.get("page_size", 16), kw.get("head_dim", 64), 8
    s = serving.KvStruct()
    s.k = s.v = FAKE
    s.layers, s.num_pages, s.kv_heads, s.page_size, s.head_dim = 1, P, H, ps, D
    s.dtype = serving.INT8MM_F16
    s.k_page_stride = s.v_page_stride = H * ps * D
    s.ks_page_stride = s.vs_page_stride = H * ps
    for n, x in kw.items():
        setattr(s, n, x)
    return ctypes.byref(s)


def test_header_binding_and_library_agree(lib):
    src = open(HEADER).read()
    fns = sorted(set(re.findall(r"INT8MM_API\s+[\w\s\*]+?\b(\w+)\s*\(", src)))
    assert fns == sorted(serving.SIGNATURES)
    for n in fns:
        assert hasattr(lib, n), n
    consts = dict(re.findall(r"#define (INT\w+) \(?(\d+(?: << \d+)?)\)?", src))
    for n in ("INT8MM_F16", "INT8MM_BF16", "INT8MM_I8", "INT4_MAX_K", "INT4_MAX_N",
              "INT4_MAX_M", "INT8MM_KV_MAX_PAGES",
              "INT8MM_KV_MAX_PAGE_SIZE", "INT8MM_KV_MAX_HEAD_DIM", "INT8MM_KV_DONE",
              "INT8MM_KV_NO_PAGES", "INT8MM_KV_BAD_ROW"):
        assert eval(consts[n]) == getattr(serving, n), n


def test_header_is_c_and_the_struct_matches(tmp_path):
    if shutil.which("gcc") is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("gcc or the ROCm headers are missing")
    fields = [n for n, _ in serving.KvStruct._fields_]
    prog = ['#include <stdio.h>', '#include <stddef.h>', '#include "int8mm_serving.h"',
            'int main(void) {', 'printf("%zu\\n", sizeof(int8mm_kv));']
    prog += [f'printf("%zu\\n", offsetof(int8mm_kv, {n}));' for n in fields] + ["return 0; }"]
    c = tmp_path / "kv.c"
    c.write_text("\n".join(prog))
    exe = str(tmp_path / "kv")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-Wno-pedantic",
                        "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-isystem",
                        "/opt/rocm/include", str(c), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    got = list(map(int, subprocess.run([exe], capture_output=True, text=True).stdout.split()))
    assert got == [ctypes.sizeof(serving.KvStruct)] + [getattr(serving.KvStruct, n).offset for n in fields]


def test_int4_sizes(lib):
    assert lib.int4_weight_bytes(64, 128) == 64 * 64
    assert lib.int4_weight_bytes(1, 1) == 16 * 64
    assert lib.int4_weight_bytes(65, 129) == 80 * 128
    assert lib.int4_param_bytes(64, 128, 128, 0) == 128
    assert lib.int4_param_bytes(64, 128, 32, 1) == 64 * 4 * 4
    assert lib.int4_param_bytes(64, 1024, 512, 0) == 64 * 8 * 2
    for g in (0, 16, 48, 96, 130, -128):
        assert lib.int4_param_bytes(64, 128, g, 0) == -1
    assert lib.int4_weight_bytes(-1, 5) == -1 and lib.int4_weight_bytes(5, (1 << 20) + 1) == -1


def _lin(lib, X=FAKE, dt=0, M=2, K=64, ldx=64, W=FAKE, p=FAKE, N=4, g=64, z=0, b=None, Y=FAKE,
         ws=None, nb=0):
    return lib.int4_linear(X, dt, M, K, ldx, W, p, N, g, z, b, Y, ws, nb, None)


def test_int4_refusals(lib):
    assert _lin(lib, dt=2) == EINVAL
    assert _lin(lib, M=-1) == ESHAPE and _lin(lib, K=-1) == ESHAPE and _lin(lib, N=-1) == ESHAPE
    assert _lin(lib, g=40) == ESHAPE and _lin(lib, ldx=63) == ESHAPE
    for n in ("X", "W", "p", "Y"):
        assert _lin(lib, **{n: None}) == EINVAL
    assert _lin(lib, X=FAKE + 1) == EINVAL and _lin(lib, W=FAKE + 8) == EINVAL
    assert _lin(lib, p=FAKE + 8) == EINVAL and _lin(lib, b=FAKE + 1) == EINVAL
    # more than 16 rows on few channels and a long K need the workspace, also
    # fewer that are not on 16 bytes
    big = dict(K=8192, ldx=8192, N=64)
    need = lib.int4_linear_workspace_size(20, 8192, 64)
    assert need >= 2 * 20 * 64 * 4
    assert _lin(lib, M=20, **big) == EWORKSPACE
    assert _lin(lib, M=20, ws=FAKE + 16, nb=1 << 30, **big) == EWORKSPACE
    assert _lin(lib, M=20, ws=FAKE, nb=need - 1, **big) == EWORKSPACE
    assert _lin(lib, X=FAKE + 2, **big) == EWORKSPACE
    assert lib.int4_linear_workspace_size(20, 1024, 64) == 0
    assert _lin(lib, M=0) == OK and _lin(lib, N=0) == OK
    assert lib.int4_pack_weight(FAKE, 4, 64, 64, FAKE, None, None, FAKE, None) == EINVAL
    assert lib.int4_pack_weight(FAKE, 4, 64, 65, FAKE, None, FAKE, FAKE, None) == ESHAPE
    assert lib.int4_pack_weight(FAKE, 4, 0, 64, None, None, None, None, None) == OK
    assert lib.int4_prepare_weight(FAKE, 2, 4, 64, 64, 0, FAKE, FAKE, None) == EINVAL
    assert lib.int4_prepare_weight(FAKE, 0, 4, 64, 64, 0, FAKE + 4, FAKE, None) == EINVAL


def _att(lib, q=FAKE, dt=0, B=2, Hq=4, qb=256, qh=64, kv=None, t=FAKE, tr=2, tw=100, n=FAKE,
         rows=None, top=1600, scale=0.1, window=0, cap=0.0, out=FAKE, lse=None, ws=FAKE,
         nb=1 << 30):
    return lib.kv_attention(q, dt, B, Hq, qb, qh, kv or _kv(), t, tr, tw, n, rows, top, scale,
                            window, cap, out, lse, ws, nb, None)


def test_attention_refusals(lib):
    for n in ("q", "t", "n", "out"):
        assert _att(lib, **{n: None}) == EINVAL, n
    assert lib.kv_attention(FAKE, 0, 2, 4, 256, 64, None, FAKE, 2, 100, FAKE, None, 1600, 0.1, 0,
                            0.0, FAKE, None, FAKE, 1 << 30, None) == EINVAL
    assert _att(lib, dt=1) == EINVAL and _att(lib, dt=2) == EINVAL
    assert _att(lib, Hq=3) == ESHAPE and _att(lib, B=-1) == ESHAPE and _att(lib, Hq=0) == ESHAPE
    assert _att(lib, window=-1) == ESHAPE and _att(lib, top=-1) == ESHAPE
    assert _att(lib, tw=1 << 27) == ESHAPE                 # positions past int32
    for bad in (math.nan, math.inf):
        assert _att(lib, scale=bad) == EINVAL and _att(lib, cap=bad) == EINVAL
    assert _att(lib, cap=-1.0) == EINVAL
    assert _att(lib, q=FAKE + 8) == EINVAL and _att(lib, qb=252) == EINVAL
    assert _att(lib, qh=60) == EINVAL and _att(lib, lse=FAKE + 2) == EINVAL
    need = lib.kv_attention_workspace_size(2, 4, 2, 64, 1600)
    assert need > 256
    assert _att(lib, ws=None) == EWORKSPACE and _att(lib, ws=FAKE + 16) == EWORKSPACE
    assert _att(lib, nb=1000) == EWORKSPACE
    assert _att(lib, B=0) == OK


def test_cache_refusals(lib):
    for kw in (dict(page_size=8), dict(page_size=24), dict(page_size=2048), dict(head_dim=72),
               dict(head_dim=272), dict(head_dim=0), dict(kv_heads=0), dict(num_pages=-1),
               dict(num_pages=(1 << 22) + 1), dict(layers=0)):
        assert _att(lib, kv=_kv(**kw), Hq=4) == ESHAPE, kw
    for kw in (dict(dtype=3), dict(k=None), dict(v=FAKE + 8), dict(k_page_stride=2047),
               dict(k_page_stride=2052), dict(v_page_stride=100), dict(dtype=2)):
        assert _att(lib, kv=_kv(**kw)) == EINVAL, kw
    i8 = dict(dtype=2, k_scale=FAKE, v_scale=FAKE)
    assert _att(lib, kv=_kv(**i8), ws=None) == EWORKSPACE  # passes up to there
    assert _att(lib, kv=_kv(**i8, ks_page_stride=33)) == EINVAL
    assert lib.kv_pages_copy(_kv(layers=2, k_layer_stride=8, v_layer_stride=1 << 20), FAKE, FAKE, 1,
                             None) == EINVAL


def test_row_and_page_refusals(lib):
    def app(k=FAKE, dt=0, T=3, kv=None, t=FAKE, tr=2, tw=4, r=FAKE, p=FAKE):
        return lib.kv_append(k, FAKE, dt, T, 128, 64, 128, 64, kv or _kv(), t, tr, tw, r, p, None)
    assert app(k=None) == EINVAL and app(t=None) == EINVAL and app(r=None) == EINVAL
    assert app(p=FAKE + 2) == EINVAL and app(dt=1) == EINVAL and app(T=-1) == ESHAPE
    assert app(tr=-1) == ESHAPE and app(tw=1 << 28) == ESHAPE
    assert app(T=0) == OK and app(kv=_kv(num_pages=0)) == OK
    assert lib.kv_gather(FAKE + 8, FAKE, 0, 3, _kv(), FAKE, 2, 4, FAKE, FAKE, None) == EINVAL
    assert lib.kv_gather(FAKE, FAKE, 1, 3, _kv(), FAKE, 2, 4, FAKE, FAKE, None) == EINVAL
    assert lib.kv_gather(FAKE, FAKE, 0, 0, _kv(), FAKE, 2, 4, FAKE, FAKE, None) == OK

    assert lib.kv_pages_copy(_kv(), None, FAKE, 1, None) == EINVAL
    assert lib.kv_pages_copy(_kv(), FAKE, FAKE, -1, None) == ESHAPE
    assert lib.kv_pages_copy(_kv(), None, None, 0, None) == OK

    def res(P=8, ps=16, t=FAKE, n=2, st=FAKE, ws=FAKE, nb=1 << 20):
        return lib.kv_pages_reserve(P, ps, t, 2, 4, FAKE, FAKE, FAKE, FAKE, n, st, ws, nb, None)
    assert res(ps=20) == ESHAPE and res(P=-1) == ESHAPE and res(n=-1) == ESHAPE
    assert res(n=16385) == ESHAPE and res(t=None) == EINVAL and res(st=None) == EINVAL
    assert res(ws=None) == EWORKSPACE and res(nb=100) == EWORKSPACE and res(n=0) == OK

    def fork(c=FAKE, ref_=FAKE, n=2, ws=FAKE, nb=1 << 20):
        return lib.kv_pages_fork(_kv(), FAKE, 2, 4, FAKE, ref_, FAKE, c, n, FAKE, ws, nb, None)
    assert fork(c=None) == EINVAL and fork(ref_=None) == EINVAL and fork(n=-1) == ESHAPE
    assert fork(ws=FAKE + 128) == EWORKSPACE and fork(nb=0) == EWORKSPACE and fork(n=0) == OK

    assert lib.kv_pages_free(8, None, 2, 4, FAKE, FAKE, FAKE, 1, None) == EINVAL
    assert lib.kv_pages_free(8, FAKE, 2, 4, FAKE, FAKE, FAKE, -1, None) == ESHAPE
    assert lib.kv_pages_free(8, FAKE, 2, 4, FAKE, FAKE, None, 0, None) == OK

    def comp(t=FAKE, out=FAKE, live=FAKE, ws=FAKE, nb=1 << 20):
        return lib.kv_pages_compact(_kv(), t, out, 2, 4, FAKE, FAKE, live, ws, nb, None)
    assert comp(t=None) == EINVAL and comp(out=None) == EINVAL and comp(live=None) == EINVAL
    assert comp(ws=None) == EWORKSPACE and comp(nb=10) == EWORKSPACE
    assert lib.kv_pages_workspace_size(-1, 1) == 0 and lib.kv_pages_workspace_size(8, 16385) == 0


def test_sizes_beyond_a_launch_are_refused(lib):
    """A launch holds fewer than 2^32 threads."""
    assert lib.int4_weight_bytes((1 << 24) + 1, 64) == -1
    assert _lin(lib, N=(1 << 24) + 1) == ESHAPE and _lin(lib, M=(1 << 21) + 1) == ESHAPE
    assert _att(lib, B=1 << 22, Hq=4) == ESHAPE and _att(lib, B=1 << 62, Hq=4) == ESHAPE
    assert lib.kv_append(FAKE, FAKE, 0, (1 << 28) + 1, 128, 64, 128, 64, _kv(), FAKE, 2, 4, FAKE,
                         FAKE, None) == ESHAPE
    assert lib.kv_gather(FAKE, FAKE, 0, (1 << 28) + 1, _kv(), FAKE, 2, 4, FAKE, FAKE, None) == ESHAPE
    assert lib.kv_pages_free(8, FAKE, 2, 4, FAKE, FAKE, FAKE, (1 << 23) + 1, None) == ESHAPE


# ---------------------------------------------- the reference, on its own terms

def test_reference_quantizers():
    g = np.random.default_rng(1)
    W = g.standard_normal((6, 70)).astype(np.float16)
    for sym in (True, False):
        c, s, z = ref.int4_quantize(W, 32, sym)
        w = ref.int4_dequant(c, s, z, 32)
        step = np.repeat(s.astype(np.float64), 32, 1)[:, :70]
        # symmetric codes reach every value within half a step; with zero
        # points the rounded zero may shift the range by half a step more
        assert np.all(np.abs(w - W) <= (0.5 if sym else 1.0) * step * (1 + 2 ** -8))
    x = g.standard_normal((5, 3, 64)).astype(np.float32)
    c, a = ref.kv_codes(x)
    assert np.all(np.abs(c * a[..., None] / 127 - x) <= a[..., None] / 254 * (1 + 1e-6))
    assert np.all(np.abs(c).max(-1) == 127)


def test_reference_attention():
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal((2, 8)), g.standard_normal((5, 8)), g.standard_normal((5, 8))
    out, lse, _, _ = ref.attention_rows(q, k, v, 0.3, 0.0)
    e = np.exp(0.3 * q @ k.T)
    assert np.allclose(out, e @ v / e.sum(1, keepdims=True)) and np.allclose(lse, np.log(e.sum(1)))
    out, lse, _, _ = ref.attention_rows(q, k[:0], v[:0], 0.3, 0.0)
    assert not out.any() and np.all(lse == -np.inf)


def test_reference_pool_keeps_its_counts():
    g = np.random.default_rng(3)
    p = ref.Pool([[-1] * 6 for _ in range(8)], [0] * 8, [0] * 30, 4)
    for step in range(60):
        rows = [int(r) for r in g.permutation(8)[:3]]
        kind = step % 4
        if kind == 0:
            p.reserve(rows, [min(24, p.lengths[r] + int(g.integers(0, 9))) for r in rows])
        elif kind == 1:
            p.fork(rows[:1], rows[1:2])
        elif kind == 2:
            p.free(rows[:1])
        else:
            live, _ = p.compact()
            assert all((r > 0) == (i < live) for i, r in enumerate(p.ref))
        count = [0] * 30
        for row, n in zip(p.table, p.lengths):
            used = -(-n // 4)
            assert all(x >= 0 for x in row[:used]) and all(x == -1 for x in row[used:])
            for x in row[:used]:
                count[x] += 1
        assert count == p.ref


def test_token_counts_at_the_limit_of_a_launch(lib):
    """The largest documented count is the last whose grid has fewer than 2^32
    threads (32 tokens a workgroup of up to 512)."""
    last = (1 << 28) - 32
    assert -(-last // 32) * 512 < 1 << 32 <= -(-(last + 1) // 32) * 512
    text = re.sub(r"\s+\*?\s*", " ", open(HEADER).read())
    assert "2^28 - 32 tokens for a kv_append or kv_gather" in text
    for T in (last + 1, 1 << 28):
        assert lib.kv_append(FAKE, FAKE, 0, T, 128, 64, 128, 64, _kv(), FAKE, 2, 4, FAKE, FAKE,
                             None) == ESHAPE
        assert lib.kv_gather(FAKE, FAKE, 0, T, _kv(), FAKE, 2, 4, FAKE, FAKE, None) == ESHAPE
    # up to there the arguments are looked at
    assert lib.kv_append(FAKE, FAKE, 0, last, 128, 64, 128, 64, _kv(), FAKE, 2, 4, FAKE, FAKE + 2,
                         None) == EINVAL
    assert lib.kv_gather(FAKE, FAKE, 0, last, _kv(), FAKE, 2, 4, FAKE, FAKE + 2, None) == EINVAL
