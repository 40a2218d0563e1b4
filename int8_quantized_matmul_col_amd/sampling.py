"""Drawing the next tokens from logits (include/int8mm_serving.h)."""

from __future__ import annotations

from typing import Union

import torch

from .binding import _check_out, _require
from .serving import (INT8MM_BF16, INT8MM_F16, INT8MM_F32, _call, _check_workspace, _lib, _on)

INT8MM_SAMPLE_MAX_V = 1 << 20
_DTYPES = {torch.float16: INT8MM_F16, torch.bfloat16: INT8MM_BF16, torch.float32: INT8MM_F32}


def _each(x, name: str, dtype, B: int, device):
    """(address or None, value): of a tensor with an entry for each row, or of
    one number for all."""
    if isinstance(x, torch.Tensor):
        if not (x.dtype is dtype and x.get_device() == device.index and x.is_contiguous()):
            _require(x, dtype, name, device)
        if x.shape != (B,):
            raise ValueError(f"{name} has shape {tuple(x.shape)}, expected [{B}]")
        return x.data_ptr(), 0
    return None, x


def sample_tokens_workspace_size(B: int, V: int) -> int:
    return int(_lib().sample_tokens_workspace_size(int(B), int(V)))


def sample_tokens(logits, u, temperature: Union[float, torch.Tensor] = 1.0,
                  top_k: Union[int, torch.Tensor] = 0, top_p: Union[float, torch.Tensor] = 1.0,
                  min_p: Union[float, torch.Tensor] = 0.0, out=None, workspace=None):
    """One token of each row: logits [B][V] (float16, bfloat16 or float32, the last
    dim contiguous), u float32 [B] uniform in [0, 1).  Returns int32 [B].

    With probabilities of logits / temperature, tokens by logit downwards and
    equal ones by index: top_k keeps the first k (0: all), top_p of these those
    with less than top_p of their mass before them, min_p those at least min_p
    times as likely as the likeliest.  The token is the first, in the
    vocabulary's order, at which the running mass of the kept exceeds u times
    all of it.  temperature 0 takes the first of the largest logits.  Each of
    the four is a number, or a tensor [B] (float32; top_k int32).  A row with NaN
    or +inf, or nothing above -inf, gives -1."""
    dt = _DTYPES.get(logits.dtype)
    if dt is None:
        raise TypeError("logits must be torch.float16, torch.bfloat16 or torch.float32, got "
                        f"{logits.dtype}")
    _on(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [B][V]")
    B, V = logits.shape
    dev = logits.device
    sb, sv = logits.stride()
    if sv != 1 and V > 1 and B > 0:
        raise ValueError("the rows of logits must be contiguous")
    if not isinstance(u, torch.Tensor):
        raise TypeError("u must be a torch.Tensor")
    u_ptr, _ = _each(u, "u", torch.float32, B, dev)
    t, t_all = _each(temperature, "temperature", torch.float32, B, dev)
    k, k_all = _each(top_k, "top_k", torch.int32, B, dev)
    p, p_all = _each(top_p, "top_p", torch.float32, B, dev)
    m, m_all = _each(min_p, "min_p", torch.float32, B, dev)
    k_all = min(max(int(k_all), 0), (1 << 31) - 1)
    if out is None:
        out = u.new_empty((B,), dtype=torch.int32)
    else:
        _check_out(out, (B,), torch.int32, "out", dev)
    if workspace is None:
        n = _lib().sample_tokens_workspace_size(B, V)
        if n:
            workspace = u.new_empty((n // 4,))
    else:
        _check_workspace(workspace, dev)
    _call("sample_tokens", dev.index, logits.data_ptr(), dt, B, V, sb, u_ptr, t, t_all, k,
          k_all, p, p_all, m, m_all, out.data_ptr(),
          None if workspace is None else workspace.data_ptr(),
          0 if workspace is None else workspace.nbytes)
    return out


__all__ = ["sample_tokens", "sample_tokens_workspace_size"]
