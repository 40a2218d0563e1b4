"""What kv_attention's probabilities carry into the sum over the values: values
that cancel, so that the result's own rounding hides nothing."""

import math

import numpy as np
import pytest
import torch

from serving_cases import DTYPES, TINY, U16, U32, dev, f64, rng

pytestmark = pytest.mark.gpu

TYPES = [("f16", "f16"), ("bf16", "bf16"), ("i8", "f16"), ("i8", "bf16")]
D, PS = 64, 16


def _probabilities(keys):
    e = np.exp(keys - keys.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def _attend(lib, cache, dtype, keys, k_scale, values, v_scale):
    """One page a sequence, one head: the scores are the keys' first dims, which
    q = (1, 0, ..) takes out exactly.  keys [B][T] and values [B][T][D] as they
    are stored (codes for int8), scales [B][T]."""
    B, T = keys.shape
    k = np.zeros((B, 1, PS, D), np.float32)
    v = np.zeros((B, 1, D, PS), np.float32)
    k[:, 0, :T, 0] = keys
    v[:, 0, :, :T] = values.transpose(0, 2, 1)
    scales = [None, None]
    if cache == "i8":
        scales = [torch.zeros((B, 1, PS), device="cuda") for _ in range(2)]
        for t, s in zip(scales, (k_scale, v_scale)):
            t[:, 0, :T] = dev(s.astype(np.float32))
    t = DTYPES.get(cache, torch.int8)
    kv = lib.PagedKV(dev(k, t), dev(v, t), *scales)
    q = torch.zeros((B, 1, D), dtype=DTYPES[dtype], device="cuda")
    q[:, 0, 0] = 1
    table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    lengths = torch.full((B,), T, dtype=torch.int32, device="cuda")
    return f64(lib.kv_attention(q, kv, table, lengths, scale=1.0)[:, 0]), q.dtype


def _error(T, top, i8):
    """Relative error of a weighted value p v / sum p in fp32, in units of u32:
    the exponent's product with log2 e (a rounded constant, one rounding) and
    its distance from the maximum (|.| <= 2 top, 6 more for float16's factor,
    one rounding), the exponential (2), both in p and in the sum; the value's
    factor of an int8 cache (4); up to T terms, the joins and the division
    (T + 16)."""
    x = top / math.log(2)
    return (2 * (math.log(2) * (1.5 * x + 2 * x + 6) + 2) + (4 if i8 else 0) + T + 16) * U32


@pytest.mark.parametrize("cache,dtype", TYPES)
def test_values_that_cancel(lib, cache, dtype):
    """The first token's values are random and the other tokens' are chosen to
    cancel what is before them as far as the cache's type goes, so the sum is a
    small part of its terms and shows the terms' errors."""
    g = rng(51)
    B, T = 512, 5
    i8 = cache == "i8"
    at = DTYPES.get(cache)
    if i8:
        keys, ks = g.integers(-127, 128, (B, T)).astype(np.float64), np.ones((B, T))
        real = keys * ks / 127
    else:
        keys = real = f64(dev(g.uniform(-1, 1, (B, T)).astype(np.float32), at))
        ks = None
    p = _probabilities(real)
    values, vs = np.zeros((B, T, D)), np.ones((B, T))
    rest, size = np.zeros((B, D)), np.zeros((B, D))
    for t in range(T):
        want = g.standard_normal((B, D)) if t == 0 else -rest / p[:, t, None]
        if i8:
            vs[:, t] = np.abs(want).max(-1).astype(np.float32)
            values[:, t] = np.rint(127 * want / vs[:, t, None]).clip(-127, 127)
            held = values[:, t] * vs[:, t, None] / 127
        else:
            values[:, t] = held = f64(dev(want.astype(np.float32), at))
        rest += p[:, t, None] * held
        size += p[:, t, None] * np.abs(held)
    assert np.median(np.abs(rest)[size > 0] / size[size > 0]) < 2.0 ** -20  # it does cancel
    got, t = _attend(lib, cache, dtype, keys, ks, values, vs)
    bound = U16[t] * np.abs(rest) + _error(T, 1.0, i8) * size + TINY[t]
    d = np.abs(got - rest)
    assert not (d > bound).any(), float((d / bound).max())
