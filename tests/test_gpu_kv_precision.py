"""What kv_attention's probabilities carry into the sum over the values: values
that cancel, so that the result's own rounding hides nothing, and a token that
dominates the softmax with a value of 0, so that what is left has small
probabilities."""

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


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("below", [8, 11, 14, 16, 17, 18, 19])
def test_small_probabilities_beside_a_token_without_value(lib, cache, dtype, below):
    """One token's score is `below` above the others', and its value is 0."""
    g = rng(52, below)
    B, T = 64, 13
    i8 = cache == "i8"
    at = DTYPES.get(cache)
    keys = np.full((B, T), -float(below)) + g.uniform(-0.5, 0.5, (B, T))
    values = g.uniform(1e4, 6e4, (B, T, D)) * g.choice([-1, 1], (B, T, D))
    keys[:, 3] = 0
    ks = vs = np.ones((B, T))
    if i8:
        ks = np.full((B, T), 20.0)
        keys = np.rint(keys * 127 / ks)
        real = keys * ks / 127
        vs = np.full((B, T), 6e4, np.float32)
        values = np.rint(127 * values / 6e4)
        held = values * vs[..., None].astype(np.float64) / 127
    else:
        keys = real = f64(dev(keys.astype(np.float32), at))
        values = held = f64(dev(values.astype(np.float32), at))
    values, held = values.copy(), held.copy()
    values[:, 3] = held[:, 3] = 0
    p = _probabilities(real)[..., None]
    want, size = (p * held).sum(1), (p * np.abs(held)).sum(1)
    got, t = _attend(lib, cache, dtype, keys, ks, values, vs)
    # float16 operands end at 2^-24: with the factors 2^6 and 2^12 at 2^-42 of
    # the largest probability, half of it in rounding
    end = 2.0 ** -43 * np.abs(held).sum(1) if cache == "f16" else 0.0
    bound = U16[t] * np.abs(want) + _error(T, below + 0.5, i8) * size + end + TINY[t]
    d = np.abs(got - want)
    assert not (d > bound * (1 + 2.0 ** -8)).any(), float((d / bound).max())
