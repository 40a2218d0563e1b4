"""Python binding of the serving operators (include/int8mm_serving.h).

As in ``binding``, every function has the name of the C entry point it calls,
checks its tensors, allocates outputs and workspaces with torch and passes
device pointers plus torch's current stream; all arithmetic runs in the HIP
kernels and there is no fallback.

* ``int4_prepare_weight`` / ``int4_pack_weight`` / ``int4_linear``: products
  of a few rows with 4-bit weights and group scales.
* ``PagedKV``: the pages of a key-value cache; ``kv_append``, ``kv_gather``,
  ``kv_attention`` work on one layer of it, ``kv_pages_*`` on its pages.
  ``kv_cache.PagedKVCache`` keeps the tables beside them.
"""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional, Tuple

import torch

from . import binding
from .binding import INT8MM_ESHAPE, Int8mmError, _check, _check_out, _require

INT8MM_F16, INT8MM_BF16, INT8MM_I8 = 0, 1, 2
INT4_MAX_K = 1 << 20
INT4_MAX_N = 1 << 24
INT4_MAX_M = 1 << 21
INT8MM_KV_MAX_PAGES = 1 << 22
INT8MM_KV_MAX_PAGE_SIZE = 1024
INT8MM_KV_MAX_HEAD_DIM = 256
INT8MM_KV_DONE, INT8MM_KV_NO_PAGES, INT8MM_KV_BAD_ROW = 0, 1, 2

_DTYPES = {torch.float16: INT8MM_F16, torch.bfloat16: INT8MM_BF16}
_CACHE_DTYPES = {**_DTYPES, torch.int8: INT8MM_I8}


class KvStruct(ctypes.Structure):
    """int8mm_kv of the C header."""
    _fields_ = (
        [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")]
        + [(n + "_layer_stride", ctypes.c_int64) for n in ("k", "v", "ks", "vs")]
        + [(n + "_page_stride", ctypes.c_int64) for n in ("k", "v", "ks", "vs")]
        + [(n, ctypes.c_int32) for n in ("layers", "num_pages", "kv_heads", "page_size",
                                         "head_dim", "dtype")])


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_INT = ctypes.c_int
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_KV = ctypes.POINTER(KvStruct)
SIGNATURES = {
    "int4_weight_bytes": (_I64, [_I64, _I64]),
    "int4_param_bytes": (_I64, [_I64, _I64, _I64, _INT]),
    "int4_pack_weight": (_INT, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P]),
    "int4_prepare_weight": (_INT, [_P, _INT, _I64, _I64, _I64, _INT, _P, _P, _P]),
    "int4_linear_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "int4_linear": (_INT, [_P, _INT, _I64, _I64, _I64, _P, _P, _I64, _I64, _INT, _P, _P, _P, _SZ,
                           _P]),
    "kv_append": (_INT, [_P, _P, _INT, _I64, _I64, _I64, _I64, _I64, _KV, _P, _I64, _I64, _P, _P,
                         _P]),
    "kv_gather": (_INT, [_P, _P, _INT, _I64, _KV, _P, _I64, _I64, _P, _P, _P]),
    "kv_attention_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I64]),
    "kv_attention": (_INT, [_P, _INT, _I64, _I64, _I64, _I64, _KV, _P, _I64, _I64, _P, _P, _I64,
                            _F, _I64, _F, _P, _P, _P, _SZ, _P]),
    "kv_pages_workspace_size": (_SZ, [_I64, _I64]),
    "kv_pages_copy": (_INT, [_KV, _P, _P, _I64, _P]),
    "kv_pages_reserve": (_INT, [_I32, _I32, _P, _I64, _I64, _P, _P, _P, _P, _I64, _P, _P, _SZ,
                                _P]),
    "kv_pages_fork": (_INT, [_KV, _P, _I64, _I64, _P, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
    "kv_pages_free": (_INT, [_I32, _P, _I64, _I64, _P, _P, _P, _I64, _P]),
    "kv_pages_compact": (_INT, [_KV, _P, _P, _I64, _I64, _P, _P, _P, _P, _SZ, _P]),
}

_fns: Optional[ctypes.CDLL] = None
_by_name: dict = {}


def _lib() -> ctypes.CDLL:
    global _fns
    if _fns is None:
        lib = binding.load()
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
            _by_name[name] = fn
        _fns = lib
    return _fns


_device = torch._C._cuda_getDevice
_stream_of = torch._C._cuda_getCurrentRawStream


def _call(name: str, index: int, *args) -> None:
    """One C call on torch's current stream of GPU `index`, with that GPU
    current (the library launches on the current one)."""
    if _fns is None:
        _lib()
    if _device() == index:
        st = _by_name[name](*args, _stream_of(index))
    else:
        with torch.cuda.device(index):
            st = _by_name[name](*args, _stream_of(index))
    if st:
        _check(name, st)


def _row_dtype(t, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {t.dtype}")
    return code


def _on(t, name: str, device=None) -> None:
    """A GPU tensor (of `device`); contiguity and type are the caller's checks."""
    if t.__class__ is torch.Tensor and t.is_cuda and (device is None
                                                      or t.get_device() == device.index):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _indexes(t, name: str, device, shape=None) -> None:
    """A contiguous int32 tensor of `device` (and shape)."""
    # one look at what is nearly always right; _require names what is wrong
    if not (t.__class__ is torch.Tensor and t.dtype is torch.int32 and t.is_contiguous()
            and t.get_device() == device.index):
        _require(t, torch.int32, name, device)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check_workspace(ws, device) -> None:
    """A caller's workspace: its bytes follow one another on `device` (the
    library looks at its size and alignment)."""
    _on(ws, "workspace", device)
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")


# ------------------------------------------------------------ 4-bit weights

class Int4Weight(NamedTuple):
    """A prepared 4-bit weight: codes and group parameters in the library's
    tile order (uint8 tensors), and what they stand for."""
    Wq: torch.Tensor
    params: torch.Tensor
    out_features: int
    in_features: int
    group_size: int
    zeros: bool


@functools.lru_cache(maxsize=None)
def _int4_bytes(N: int, K: int, group: int, zeros: bool) -> Tuple[int, int]:
    """int4_weight_bytes and int4_param_bytes (-1 where there is no such weight)."""
    lib = _lib()
    return lib.int4_weight_bytes(N, K), lib.int4_param_bytes(N, K, group, int(zeros))


def _int4_buffers(N: int, K: int, group: int, zeros: bool, device) -> Tuple:
    nw, np_ = _int4_bytes(N, K, group, zeros)
    if nw < 0 or np_ < 0:
        raise Int8mmError("int4_weight_bytes", INT8MM_ESHAPE)
    return (torch.empty((nw,), dtype=torch.uint8, device=device),
            torch.empty((np_,), dtype=torch.uint8, device=device))


def int4_pack_weight(codes, scales, zeros=None, group_size: int = 128) -> Int4Weight:
    """Already-quantized codes into the prepared form: codes uint8 [N][K]
    (0..15), scales float16 [N][ceil(K/group_size)], zeros uint8 of the same
    shape or None (8): the weight is (codes - zeros) * scales per group.
    group_size: 32, 64 or a multiple of 128."""
    _require(codes, torch.uint8, "codes")
    if codes.dim() != 2:
        raise ValueError("codes must be 2-D [N][K]")
    N, K = codes.shape
    g = int(group_size)
    Wq, params = _int4_buffers(N, K, g, zeros is not None, codes.device)
    shape = (N, (K + g - 1) // g)
    for t, dt, name in ((scales, torch.float16, "scales"), (zeros, torch.uint8, "zeros")):
        if t is None and name == "zeros":
            continue
        _require(t, dt, name, codes.device)
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    _call("int4_pack_weight", codes.device.index, codes.data_ptr(), N, K, g, scales.data_ptr(),
          None if zeros is None else zeros.data_ptr(), Wq.data_ptr(), params.data_ptr())
    return Int4Weight(Wq, params, N, K, g, zeros is not None)


def int4_prepare_weight(W, group_size: int = 128, symmetric: bool = True) -> Int4Weight:
    """One-time 4-bit quantization of W (float16 or bfloat16 [N][K]) per output
    channel and group of group_size inputs: symmetric (max|w|/7) or with zero
    points ((max - min)/15)."""
    dt = _row_dtype(W, "W")
    _require(W, W.dtype, "W")
    if W.dim() != 2:
        raise ValueError("W must be 2-D [N][K]")
    N, K = W.shape
    g = int(group_size)
    Wq, params = _int4_buffers(N, K, g, not symmetric, W.device)
    _call("int4_prepare_weight", W.device.index, W.data_ptr(), dt, N, K, g, int(not symmetric),
          Wq.data_ptr(), params.data_ptr())
    return Int4Weight(Wq, params, N, K, g, not symmetric)


def int4_unpack_weight(w: Int4Weight) -> Tuple:
    """(codes uint8 [N][K], scales float16 [N][groups], zeros uint8 or None) of
    a prepared weight: the reverse of int4_pack_weight (an index permutation)."""
    N, K, g = w.out_features, w.in_features, w.group_size
    nt, gs = (K + 127) // 128, min(g, 128)
    Np = (N + 15) // 16 * 16
    dev = w.Wq.device
    if N == 0 or K == 0:
        shape = (N, (K + g - 1) // g)
        return (torch.empty((N, K), dtype=torch.uint8, device=dev),
                torch.empty(shape, dtype=torch.float16, device=dev),
                torch.empty(shape, dtype=torch.uint8, device=dev) if w.zeros else None)
    # [panel][tile][lane = 16*q + r][dword j][byte] -> nibbles at 2*byte + half
    b = w.Wq.view(Np // 16, nt, 4, 16, 4, 4)
    nib = torch.stack((b & 15, b >> 4), -1).flatten(-2)           # [.., 8] by bit position
    nib = nib[..., [0, 4, 1, 5, 2, 6, 3, 7]]                        # element e at p(e)
    codes = nib.permute(0, 3, 1, 4, 2, 5).reshape(Np, nt * 128)    # k = 32 j + 8 q + e
    par = w.params.view(torch.float16).view(Np // 16, nt, 16, 128 // gs, 2 if w.zeros else 1)
    par = par.permute(0, 2, 1, 3, 4).reshape(Np, nt * (128 // gs), -1)[:N, ::g // gs]
    par = par[:, : (K + g - 1) // g]
    return (codes[:N, :K].contiguous(), par[..., 0].contiguous(),
            (par[..., 1] - 1024).to(torch.uint8).contiguous() if w.zeros else None)


def _check_weight(w: Int4Weight, device) -> None:
    """Whether a weight's buffers lie on `device` and are what its fields say."""
    for t, name in ((w.Wq, "Wq"), (w.params, "params")):
        _require(t, torch.uint8, name, device)
    sizes = _int4_bytes(*w[2:])
    if min(sizes) < 0:
        raise Int8mmError("int4_linear", INT8MM_ESHAPE)
    if (w.Wq.numel(), w.params.numel()) != sizes:
        raise ValueError(
            f"the weight's buffers have {w.Wq.numel()} and {w.params.numel()} bytes, not the "
            f"{sizes[0]} and {sizes[1]} of {w.out_features} x {w.in_features} codes in groups of "
            f"{w.group_size}{' with zero points' if w.zeros else ''}")


def int4_linear_workspace_size(M: int, K: int, N: int) -> int:
    return int(_lib().int4_linear_workspace_size(int(M), int(K), int(N)))


def int4_linear(X, w: Int4Weight, bias=None, out=None, workspace=None):
    """Y = X (codes - zeros)^T * scales (+ bias): X float16 or bfloat16 [M][K]
    (rows may be strided), bias [N] of the same type or None.  Returns [M][N]
    of X's type, rounded once.  Meant for few rows (M up to 64 reads the weight
    once)."""
    dt = _DTYPES.get(X.dtype)
    index = X.get_device()
    if dt is None or index < 0:
        _row_dtype(X, "X")
        _on(X, "X")
    Wq, params, N, K, group, zeros = w
    shape = X.shape
    if len(shape) != 2 or shape[1] != K:
        raise ValueError(f"X has shape {tuple(shape)}, expected [M][{K}]")
    # the buffers are read by what the fields say: one look at what is nearly
    # always right
    if not (Wq.__class__ is params.__class__ is torch.Tensor
            and Wq.get_device() == params.get_device() == index
            and (Wq.numel(), params.numel()) == _int4_bytes(N, K, group, zeros)
            and Wq.is_contiguous() and params.is_contiguous()):
        _check_weight(w, X.device)
    M = shape[0]
    if M > 0 and K > 1 and X.stride(1) != 1:
        raise ValueError("the rows of X must be contiguous")
    ldx = X.stride(0) if M > 1 else K
    if ldx < K:
        raise ValueError("the rows of X must not overlap")
    if bias is not None:
        _require(bias, X.dtype, "bias", X.device)
        if bias.numel() != N:
            raise ValueError(f"bias has {bias.numel()} entries, expected {N}")
    if out is None:
        Y = X.new_empty((M, N))
    else:
        _check_out(out, (M, N), X.dtype, "out", X.device)
        Y = out
    # up to 16 rows on 16 bytes need no workspace
    if workspace is None and (M > 16 or K % 8 or ldx % 8 or X.data_ptr() % 16):
        n = _lib().int4_linear_workspace_size(M, K, N)
        if n:
            workspace = X.new_empty((n // 4,), dtype=torch.float32)
    elif workspace is not None:
        _check_workspace(workspace, X.device)
    _call("int4_linear", index, X.data_ptr(), dt, M, K, ldx, Wq.data_ptr(), params.data_ptr(), N,
          group, zeros, None if bias is None else bias.data_ptr(), Y.data_ptr(),
          None if workspace is None else workspace.data_ptr(),
          0 if workspace is None else workspace.nbytes)
    return Y


# ---------------------------------------------------------- key-value pages

class PagedKV:
    """The pages of a key-value cache: k [pages][kv_heads][page_size][head_dim],
    v [pages][kv_heads][head_dim][page_size] (float16, bfloat16 or int8), and for
    int8 the scales k_scale, v_scale float32 [pages][kv_heads][page_size]; all
    with a leading [layers] for a whole cache.  The dims of one page are
    contiguous.  Holds the tensors; copies nothing."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        _on(k, "k")
        dev = k.device
        _on(v, "v", dev)
        dt = _CACHE_DTYPES.get(k.dtype)
        if dt is None:
            raise TypeError(f"a cache is torch.float16, torch.bfloat16 or torch.int8, got {k.dtype}")
        if v.dtype != k.dtype:
            raise TypeError(f"v must be {k.dtype}, got {v.dtype}")
        if k.dim() not in (4, 5) or v.dim() != k.dim():
            raise ValueError("k and v are [pages][heads][..][..], or [layers] of that")
        *lead, ps, D = k.shape
        if tuple(v.shape) != (*lead, D, ps):
            raise ValueError(f"v has shape {tuple(v.shape)}, expected {(*lead, D, ps)}")
        if (dt == INT8MM_I8) != (k_scale is not None) or (k_scale is None) != (v_scale is None):
            raise ValueError("an int8 cache has k_scale and v_scale, another has neither")
        named = [("k", k), ("v", v)]
        if k_scale is not None:
            for n, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                _on(t, n, dev)
                if t.dtype != torch.float32:
                    raise TypeError(f"{n} must be torch.float32, got {t.dtype}")
                if tuple(t.shape) != (*lead, ps):
                    raise ValueError(f"{n} has shape {tuple(t.shape)}, expected {(*lead, ps)}")
                named.append((n, t))
        layered = k.dim() == 5
        pages, heads = lead[-2], lead[-1]
        s = KvStruct()
        for n, t in named:
            inner = t[0, 0] if layered and t.shape[0] and pages else t[0] if pages and not layered else None
            if inner is not None and not inner.is_contiguous():
                raise ValueError(f"the dims of one page of {n} must be contiguous")
            short = {"k_scale": "ks", "v_scale": "vs"}.get(n, n)
            setattr(s, n, t.data_ptr())
            setattr(s, short + "_page_stride", self._stride(t, 1 if layered else 0))
            setattr(s, short + "_layer_stride", self._stride(t, 0) if layered else 0)
        s.layers = k.shape[0] if layered else 1
        s.num_pages, s.kv_heads, s.page_size, s.head_dim, s.dtype = pages, heads, ps, D, dt
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.layered = layered
        self.layers, self.num_pages, self.kv_heads = s.layers, pages, heads
        self.page_size, self.head_dim, self.dtype, self.device = ps, D, k.dtype, dev
        self.index = dev.index
        # the types of rows beside this cache
        self._rows = dict(_DTYPES) if dt == INT8MM_I8 else {k.dtype: dt}
        self._struct = s
        self._ref = ctypes.byref(s)

    @staticmethod
    def _stride(t, dim: int) -> int:
        if t.shape[dim] > 1:
            return t.stride(dim)
        n = 1  # the distance of a single layer or page is never used
        for d in t.shape[dim + 1:]:
            n *= d
        return n

    def layer(self, i: int) -> "PagedKV":
        """One layer's pages."""
        if not self.layered:
            raise ValueError("these are the pages of one layer")
        return PagedKV(self.k[i], self.v[i], None if self.k_scale is None else self.k_scale[i],
                       None if self.v_scale is None else self.v_scale[i])

    def row_dtype(self, dtype, name: str) -> int:
        """Code of the rows' type beside this cache."""
        code = self._rows.get(dtype)
        if code is None:
            want = "torch.float16 or torch.bfloat16" if self.dtype == torch.int8 else self.dtype
            raise TypeError(f"{name} must be {want}, got {dtype}")
        return code


def _one_layer(kv: PagedKV) -> None:
    if kv.__class__ is PagedKV and not kv.layered:
        return
    if not isinstance(kv, PagedKV):
        raise TypeError("kv must be a PagedKV")
    if kv.layered:
        raise ValueError("kv must be one layer's pages (see PagedKV.layer)")


def _check_table(table, device) -> None:
    _indexes(table, "table", device)
    if table.dim() != 2:
        raise ValueError("table must be 2-D [rows][pages]")


def kv_append(k, v, kv: PagedKV, table, rows, positions) -> None:
    """Writes T tokens' keys and values (k, v [T][kv_heads][head_dim], last dim
    contiguous) to positions int32 [T] of the sequences in table rows int32
    [T], quantized for an int8 cache.  Tokens whose place does not exist are
    skipped.  The pages have to be there (kv_pages_reserve)."""
    _one_layer(kv)
    dev = kv.device
    dt = kv.row_dtype(k.dtype, "k")
    _on(k, "k", dev)
    _on(v, "v", dev)
    if v.dtype != k.dtype:
        raise TypeError(f"v must be {k.dtype}, got {v.dtype}")
    shape = (positions.numel(), kv.kv_heads, kv.head_dim)
    if k.shape != shape or v.shape != shape:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)}: expected {shape}")
    (kt, kh, kd), (vt, vh, vd) = k.stride(), v.stride()
    if kd != 1 or vd != 1:
        raise ValueError("the last dim of k and v must be contiguous")
    _check_table(table, dev)
    _indexes(rows, "rows", dev, shape[:1])
    _indexes(positions, "positions", dev, shape[:1])
    _call("kv_append", kv.index, k.data_ptr(), v.data_ptr(), dt, shape[0], kt, kh, vt, vh, kv._ref, table.data_ptr(), table.shape[0], table.shape[1],
          rows.data_ptr(), positions.data_ptr())


def kv_gather(kv: PagedKV, table, rows, positions, dtype=None, out=None) -> Tuple:
    """The keys and values at T (row, position) places as contiguous
    [T][kv_heads][head_dim] tensors (zeros where there is no such place).
    dtype: the cache's own; float16 (default) or bfloat16 for an int8 cache."""
    _one_layer(kv)
    dev = kv.device
    if dtype is None:
        dtype = torch.float16 if kv.dtype == torch.int8 else kv.dtype
    dt = kv.row_dtype(dtype, "dtype")
    _check_table(table, dev)
    T = positions.numel()
    _indexes(rows, "rows", dev, (T,))
    _indexes(positions, "positions", dev, (T,))
    shape = (T, kv.kv_heads, kv.head_dim)
    if out is None:
        k = kv.k.new_empty(shape, dtype=dtype)
        v = kv.k.new_empty(shape, dtype=dtype)
    else:
        k, v = out
        _check_out(k, shape, dtype, "out[0] (k)", dev)
        _check_out(v, shape, dtype, "out[1] (v)", dev)
    _call("kv_gather", kv.index, k.data_ptr(), v.data_ptr(), dt, T, kv._ref, table.data_ptr(),
          table.shape[0], table.shape[1], rows.data_ptr(), positions.data_ptr())
    return k, v


def kv_attention_workspace_size(B: int, q_heads: int, kv_heads: int, head_dim: int,
                                max_len: int) -> int:
    return int(_lib().kv_attention_workspace_size(int(B), int(q_heads), int(kv_heads),
                                                  int(head_dim), int(max_len)))


def kv_attention(q, kv: PagedKV, table, lengths, rows=None, scale: Optional[float] = None,
                 window: int = 0, softcap: float = 0.0, max_len: Optional[int] = None,
                 return_lse: bool = False, out=None, workspace=None):
    """Attention of one new token per sequence: q [B][q_heads][head_dim] over
    the first lengths[row] tokens of the sequences in table rows `rows` int32
    [B] (None: 0 .. B-1), the last `window` of them if window > 0.

    scale defaults to head_dim ** -0.5; softcap c > 0 caps the scores at
    c * tanh(s / c); max_len is an upper bound of the lengths that the host
    knows (default: what the table holds).  Returns out [B][q_heads][head_dim]
    of q's type, with return_lse also log-sum-exp float32 [B][q_heads].  A
    sequence without visible tokens gives 0 and -inf.  Above 256 visible tokens
    other rows' lengths may change how a row's sums are rounded."""
    _one_layer(kv)
    dev = kv.device
    dt = kv.row_dtype(q.dtype, "q")
    _on(q, "q", dev)
    shape = q.shape
    if len(shape) != 3 or shape[2] != kv.head_dim:
        raise ValueError(f"q has shape {tuple(shape)}, expected [B][q_heads][{kv.head_dim}]")
    B, Hq, D = shape
    if Hq == 0 or Hq % kv.kv_heads:
        raise ValueError(f"{Hq} query heads do not divide over {kv.kv_heads} kv heads")
    sb, sh, sd = q.stride()
    if sd != 1 or sb % 8 or sh % 8 or q.data_ptr() % 16:
        # (contiguous() leaves a view alone whose odd strides are of single rows)
        q = q.contiguous()
        if q.data_ptr() % 16:
            q = q.clone(memory_format=torch.contiguous_format)
        sb, sh = Hq * D, D
    _check_table(table, dev)
    S, width = table.shape
    _indexes(lengths, "lengths", dev, (S,))
    if rows is not None:
        _indexes(rows, "rows", dev, (B,))
    elif B > S:
        raise ValueError(f"{B} queries, and the table has {S} rows")
    room = width * kv.page_size
    max_len = room if max_len is None else min(int(max_len), room)
    if out is None:
        out = q.new_empty(shape)
    else:
        _check_out(out, (B, Hq, D), q.dtype, "out", dev)
    lse = q.new_empty((B, Hq), dtype=torch.float32) if return_lse else None
    if workspace is None:
        n = _lib().kv_attention_workspace_size(B, Hq, kv.kv_heads, D, max_len)
        if n:
            workspace = table.new_empty((n // 4,))
    else:
        _check_workspace(workspace, dev)
    _call("kv_attention", kv.index, q.data_ptr(), dt, B, Hq, sb, sh, kv._ref,
          table.data_ptr(), S, width, lengths.data_ptr(),
          None if rows is None else rows.data_ptr(), max_len,
          D ** -0.5 if scale is None else scale, window, softcap, out.data_ptr(),
          None if lse is None else lse.data_ptr(),
          None if workspace is None else workspace.data_ptr(),
          0 if workspace is None else workspace.nbytes)
    return (out, lse) if return_lse else out


def _pages_args(table, lengths, refcount, num_pages, device) -> None:
    _check_table(table, device)
    if lengths is not None:
        _indexes(lengths, "lengths", device, (table.shape[0],))
    _indexes(refcount, "refcount", device, (num_pages,) if num_pages is not None else None)


def _pages_workspace(num_pages: int, n: int, device, workspace) -> torch.Tensor:
    if workspace is not None:
        _check_workspace(workspace, device)
        return workspace
    size = _lib().kv_pages_workspace_size(num_pages, n)
    if size == 0:
        raise Int8mmError("kv_pages_workspace_size", INT8MM_ESHAPE)
    return torch.empty((size,), dtype=torch.uint8, device=device)


def kv_pages_copy(kv: PagedKV, src, dst) -> None:
    """Page dst[i] becomes a copy of page src[i] (int32 [n]), every layer.
    Pairs with an id out of range are skipped; a destination must not appear
    twice, nor as a source."""
    _indexes(src, "src", kv.device)
    _indexes(dst, "dst", kv.device, src.shape)
    _call("kv_pages_copy", kv.index, kv._ref, src.data_ptr(), dst.data_ptr(), src.numel())


def kv_pages_reserve(table, lengths, refcount, rows, new_lengths, page_size: int, workspace=None):
    """Grows sequences to new_lengths[i] tokens: table row rows[i] gets the
    pages it lacks, lowest free ids first, and its length is set.  Returns
    int32 [n]: INT8MM_KV_DONE, _NO_PAGES (unchanged) or _BAD_ROW."""
    dev = table.device
    _pages_args(table, lengths, refcount, None, dev)
    if refcount.dim() != 1:
        raise ValueError("refcount must be 1-D")
    _indexes(rows, "rows", dev)
    _indexes(new_lengths, "new_lengths", dev, rows.shape)
    n, P = rows.numel(), refcount.numel()
    status = rows.new_empty(rows.shape)
    ws = _pages_workspace(P, n, dev, workspace)
    _call("kv_pages_reserve", dev.index, P, page_size, table.data_ptr(), table.shape[0], table.shape[1],
          lengths.data_ptr(), refcount.data_ptr(), rows.data_ptr(), new_lengths.data_ptr(), n,
          status.data_ptr(), ws.data_ptr(), ws.nbytes)
    return status


def kv_pages_fork(kv: PagedKV, table, lengths, refcount, parents, children, workspace=None):
    """children[i] (an empty row) becomes a sequence with parents[i]'s tokens:
    whole pages shared, a partly filled last page copied (every layer of kv)
    into the lowest free one.  Returns int32 [n] as kv_pages_reserve."""
    dev = kv.device
    _pages_args(table, lengths, refcount, kv.num_pages, dev)
    _indexes(parents, "parents", dev)
    _indexes(children, "children", dev, parents.shape)
    n = parents.numel()
    status = parents.new_empty(parents.shape)
    ws = _pages_workspace(kv.num_pages, n, dev, workspace)
    _call("kv_pages_fork", kv.index, kv._ref, table.data_ptr(), table.shape[0], table.shape[1],
          lengths.data_ptr(), refcount.data_ptr(), parents.data_ptr(), children.data_ptr(), n,
          status.data_ptr(), ws.data_ptr(), ws.nbytes)
    return status


def kv_pages_free(table, lengths, refcount, rows) -> None:
    """Counts the pages of the sequences in table rows `rows` down (0: free),
    sets the rows to -1 and their lengths to 0."""
    dev = table.device
    _pages_args(table, lengths, refcount, None, dev)
    _indexes(rows, "rows", dev)
    _call("kv_pages_free", dev.index, refcount.numel(), table.data_ptr(), table.shape[0], table.shape[1],
          lengths.data_ptr(), refcount.data_ptr(), rows.data_ptr(), rows.numel())


def kv_pages_compact(kv: PagedKV, table, refcount, out: Optional[Tuple] = None, workspace=None):
    """Moves the used pages (every layer) into the low ids and renames them in
    the table.  Returns (table, refcount, n_live int32 [1]); the first two are
    changed in place, or written to out = (table, refcount)."""
    dev = kv.device
    _pages_args(table, None, refcount, kv.num_pages, dev)
    t, r = (table, refcount) if out is None else out
    if out is not None:
        _check_out(t, table.shape, torch.int32, "out[0] (table)", dev)
        _check_out(r, refcount.shape, torch.int32, "out[1] (refcount)", dev)
    n_live = table.new_empty((1,))
    ws = _pages_workspace(kv.num_pages, 0, dev, workspace)
    _call("kv_pages_compact", kv.index, kv._ref, table.data_ptr(), t.data_ptr(), table.shape[0],
          table.shape[1], refcount.data_ptr(), r.data_ptr(), n_live.data_ptr(), ws.data_ptr(),
          ws.nbytes)
    return t, r, n_live
