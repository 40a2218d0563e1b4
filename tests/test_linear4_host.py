"""Int4Linear's state (no GPU): the bytes of a prepared weight do not say what
they are, so the state does, and loading asks."""

import copy

import pytest

torch = pytest.importorskip("torch")

from int8_quantized_matmul_col_amd import Int4Linear, Int4Weight  # noqa: E402


def _layer(N=32, K=256, group=128, zeros=False, bias=False, fill=0):
    nt, panels = (K + 127) // 128, (N + 15) // 16
    entry = 128 // min(group, 128) * (4 if zeros else 2)
    w = Int4Weight(torch.full((panels * nt * 1024,), fill, dtype=torch.uint8),
                   torch.full((panels * nt * 16 * entry,), fill, dtype=torch.uint8), N, K, group, zeros)
    return Int4Linear(w, torch.full((N,), fill, dtype=torch.float16) if bias else None)


@pytest.mark.parametrize("kw", [
    dict(group=64), dict(group=128, zeros=True), dict(group=32, zeros=True), dict(group=256, bias=True)])
def test_state_goes_round(kw):
    a, b = _layer(fill=7, **kw), _layer(fill=1, **kw)
    b.load_state_dict(a.state_dict())
    for x, y in zip(a.state_dict().values(), b.state_dict().values()):
        assert torch.equal(x, y)
    assert torch.equal(copy.deepcopy(a).Wq, a.Wq)


@pytest.mark.parametrize("saved,layer", [
    (dict(group=64), dict(group=128, zeros=True)),      # the same bytes, read otherwise
    (dict(group=128, zeros=True), dict(group=64)),
    (dict(group=32), dict(group=64, zeros=True)),
    (dict(group=128), dict(group=256)),
    (dict(K=250), dict(K=256)),
    (dict(N=30), dict(N=32)),
])
def test_another_format_is_refused(saved, layer):
    a, b = _layer(fill=7, **saved), _layer(fill=1, **layer)
    assert a.Wq.shape == b.Wq.shape and a.params.shape == b.params.shape
    before = {n: t.clone() for n, t in b.state_dict().items()}
    for strict in (True, False):
        with pytest.raises(RuntimeError, match="group_size"):
            b.load_state_dict(a.state_dict(), strict=strict)
        for n, t in b.state_dict().items():
            assert torch.equal(t, before[n]), n


def test_state_of_a_model_and_of_before():
    """Layers inside a model; and a state that was saved without the format."""
    a = torch.nn.Sequential(_layer(group=64, fill=3), torch.nn.ReLU(), _layer(N=16, K=32, bias=True, fill=5))
    b = torch.nn.Sequential(_layer(group=64), torch.nn.ReLU(), _layer(N=16, K=32, bias=True))
    b.load_state_dict(a.state_dict())
    assert torch.equal(b[0].Wq, a[0].Wq) and torch.equal(b[2].bias, a[2].bias)
    old = {n: t for n, t in a.state_dict().items() if n.rsplit(".", 1)[1] in ("Wq", "params", "bias")}
    assert len(old) == 5
    c = torch.nn.Sequential(_layer(group=64), torch.nn.ReLU(), _layer(N=16, K=32, bias=True))
    missing = c.load_state_dict(old)
    assert not missing.missing_keys and not missing.unexpected_keys
    assert torch.equal(c[2].params, a[2].params)
    b[0] = _layer(group=128, zeros=True)
    with pytest.raises(RuntimeError, match="0: .*group_size"):
        b.load_state_dict(a.state_dict())
