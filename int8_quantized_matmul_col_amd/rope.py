"""Rotary positions: the frequencies of a model, and queries and keys turned by
them with each head's norm in the same pass (include/int8mm_serving.h).

    turning = mm.rotary(128, theta=10000.0)                # once a model
    q, k = mm.qk_rope(q, k, positions, turning, q_weight, k_weight)
"""

from __future__ import annotations

import math
from typing import NamedTuple, Optional, Sequence, Tuple, Union

import torch

from .binding import _require
from .serving import _DTYPES, _call, _indexes, _on, _row_dtype

INT8MM_ROPE_MAX_DIM = 256
INT8MM_ROPE_HALF, INT8MM_ROPE_INTERLEAVED = 0, 1
_LAYOUTS = {"half": INT8MM_ROPE_HALF, "interleaved": INT8MM_ROPE_INTERLEAVED}


class Rotary(NamedTuple):
    """Prepared frequencies: turns (int64 [rot_dim / 2], 64-bit fractions of a
    turn per position), the layout of the pairs and the factor on what is
    turned."""
    turns: torch.Tensor
    rot_dim: int
    layout: int
    factor: float


def rotary_frequencies(rot_dim: int, theta: float = 10000.0, scaling: Optional[str] = None,
                       factor: float = 1.0, original_len: int = 0, low: float = 1.0,
                       high: float = 32.0) -> torch.Tensor:
    """Radians per position, float64 [rot_dim / 2]: theta ** (-2 i / rot_dim), and
    for a context `factor` times as long as trained

    * "linear": divided by factor;
    * "ntk": theta times factor ** (rot_dim / (rot_dim - 2)), so that the slowest
      pair is divided by factor and the fastest kept;
    * "parts": with r the turns that a pair makes in original_len positions, kept
      for r >= high, divided by factor for r <= low, in between mixed linearly
      in r."""
    if rot_dim < 0 or rot_dim > INT8MM_ROPE_MAX_DIM or rot_dim % 2:
        raise ValueError(f"rot_dim must be even, 0 to {INT8MM_ROPE_MAX_DIM}, got {rot_dim}")
    if not (theta > 0 and factor > 0 and math.isfinite(theta) and math.isfinite(factor)):
        raise ValueError("theta and factor must be positive")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    if scaling == "ntk" and rot_dim > 2:
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    inv = theta ** (-2.0 * i / max(rot_dim, 1))
    if scaling in (None, "ntk"):
        return inv
    if scaling == "linear":
        return inv / factor
    if scaling == "parts":
        if original_len < 1 or not high > low:
            raise ValueError("\"parts\" takes original_len > 0 and high > low")
        keep = ((original_len * inv / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        return inv / factor * (1 - keep) + inv * keep
    raise ValueError(f"scaling is None, \"linear\", \"ntk\" or \"parts\", got {scaling!r}")


def rope_prepare(inv_freq) -> torch.Tensor:
    """Frequencies in radians per position (float64 [n], on the GPU, below 2^20)
    as 64-bit fractions of a turn, int64 [n]."""
    _require(inv_freq, torch.float64, "inv_freq")
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be 1-D")
    turns = torch.empty(inv_freq.shape, dtype=torch.int64, device=inv_freq.device)
    _call("rope_prepare", inv_freq.device.index, inv_freq.data_ptr(), inv_freq.numel(),
          turns.data_ptr())
    return turns


def rotary(rot_dim: int, theta: float = 10000.0, layout: str = "half",
           scaling: Optional[str] = None, factor: float = 1.0, original_len: int = 0,
           low: float = 1.0, high: float = 32.0, attention_factor: float = 1.0,
           inv_freq: Optional[Union[torch.Tensor, Sequence[float]]] = None,
           device="cuda") -> Rotary:
    """A model's rotation of the first rot_dim dims of each head, made once.

    layout "half" pairs dims i and rot_dim / 2 + i, "interleaved" 2 i and 2 i + 1.
    The frequencies are those of rotary_frequencies, or inv_freq (radians per
    position, rot_dim / 2 of them).  attention_factor multiplies what is turned."""
    if layout not in _LAYOUTS:
        raise ValueError(f"layout is \"half\" or \"interleaved\", got {layout!r}")
    if not math.isfinite(attention_factor):
        raise ValueError("attention_factor must be finite")
    if inv_freq is None:
        inv = rotary_frequencies(rot_dim, theta, scaling, factor, original_len, low, high)
    else:
        inv = torch.as_tensor(inv_freq, dtype=torch.float64).detach().reshape(-1).cpu()
        if rot_dim != 2 * inv.numel() or rot_dim > INT8MM_ROPE_MAX_DIM:
            raise ValueError(f"{inv.numel()} frequencies for rot_dim {rot_dim}")
    if not bool((inv.abs() < 2.0 ** 20).all()):
        raise ValueError("frequencies must be below 2^20 radians a position")
    return Rotary(rope_prepare(inv.to(device)), int(rot_dim), _LAYOUTS[layout],
                  float(attention_factor))


def _rows(t, name: str, T: int, D: Optional[int], device):
    """(heads, token distance, head distance) of rows [T][heads][D]."""
    _on(t, name, device)
    if t.dim() != 3 or t.shape[0] != T or t.shape[2] != D:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [{T}][heads][{D}]")
    st, sh, sd = t.stride()
    if sd != 1 and D > 1 and t.numel() > 0:
        raise ValueError(f"the last dim of {name} must be contiguous")
    return t.shape[1], st, sh


def _check_weight(w, name: str, dtype, D: int, device) -> None:
    _require(w, dtype, name, device)
    if w.shape != (D,):
        raise ValueError(f"{name} has shape {tuple(w.shape)}, expected [{D}]")


def qk_rope(q, k, positions, rotary: Rotary, q_weight=None, k_weight=None, eps: float = 1e-6,
            out: Optional[Tuple] = None) -> Tuple:
    """Queries and keys [T][heads][head_dim] (float16 or bfloat16, the last dim
    contiguous, other strides any; k may be None) turned by positions int32
    [T], after x * (mean(x^2) + eps)^(-1/2) * weight over each head's dims where
    there is a weight [head_dim].  fp32 inside, rounded once.

    Returns new contiguous (q, k), or writes out = (q, k), which may be the
    inputs themselves."""
    dtype = q.dtype
    dt = _DTYPES.get(dtype)
    index = q.get_device()
    dev = q.device
    if dt is None or index < 0:
        _row_dtype(q, "q")
        _on(q, "q")
    if q.dim() != 3:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [T][heads][head_dim]")
    T, _, D = q.shape
    Hq, qt, qh = _rows(q, "q", T, D, dev)
    Hk = kt = kh = 0
    if k is not None:
        if k.dtype is not dtype:
            raise TypeError(f"k must be {dtype}, got {k.dtype}")
        Hk, kt, kh = _rows(k, "k", T, D, dev)
    _indexes(positions, "positions", dev, (T,))
    if rotary.__class__ is not Rotary:
        raise TypeError("rotary must be a Rotary (see rotary())")
    turns, rot_dim, layout, factor = rotary
    if not (turns.dtype is torch.int64 and turns.get_device() == index and turns.is_contiguous()):
        _require(turns, torch.int64, "rotary.turns", dev)
    if turns.numel() * 2 != rot_dim or rot_dim > D:
        raise ValueError(f"{turns.numel()} frequencies of rot_dim {rot_dim} for heads of {D} dims")
    if q_weight is not None:
        _check_weight(q_weight, "q_weight", dtype, D, dev)
    if k_weight is not None:
        _check_weight(k_weight, "k_weight", dtype, D, dev)
    if out is None:
        yq = q.new_empty((T, Hq, D))
        yk = None if k is None else q.new_empty((T, Hk, D))
        qot, qoh, kot, koh = Hq * D, D, Hk * D, D
    else:
        yq, yk = out
        if yq.dtype != dtype or (yk is None) != (k is None) or (yk is not None and yk.dtype != dtype):
            raise TypeError(f"out must be tensors of {dtype} for q and for k, if there is one")
        n, qot, qoh = _rows(yq, "out[0] (q)", T, D, dev)
        m, kot, koh = (0, 0, 0) if yk is None else _rows(yk, "out[1] (k)", T, D, dev)
        if (n, m) != (Hq, Hk):
            raise ValueError(f"out has {n} and {m} heads, expected {Hq} and {Hk}")
    _call("qk_rope", index, q.data_ptr(), None if k is None else k.data_ptr(), dt, T, Hq, Hk,
          D, qt, qh, kt, kh, positions.data_ptr(), turns.data_ptr(), rot_dim, layout, factor,
          None if q_weight is None else q_weight.data_ptr(),
          None if k_weight is None else k_weight.data_ptr(), eps, yq.data_ptr(),
          None if yk is None else yk.data_ptr(), qot, qoh, kot, koh)
    return yq, yk


__all__ = ["Rotary", "qk_rope", "rope_prepare", "rotary", "rotary_frequencies"]
