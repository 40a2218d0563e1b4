"""The decoding example runs, and agrees with the same model run densely."""

import importlib.util
import os

import pytest

pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                     "serve.py")

# Relative to the logits' rms.  A sum rounded otherwise moves an activation by
# a few 2^-11 and may so move an int8 code by one step: a row's codes carry a
# noise of about 3.5/127/sqrt(12) = 0.8%, of which few codes take part.  One
# layer's whole noise, 4 of its deviations out: 0.03.  int8 pages add such a
# noise to keys and values of two layers, in full: 0.008 * 2 * 4.5 = 0.07.
TOLERANCE = {"f16": 0.03, "i8": 0.1}


@pytest.mark.parametrize("cache", ["f16", "i8"])
def test_example(cache):
    spec = importlib.util.spec_from_file_location("serve_example", _PATH)
    serve = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(serve)
    assert serve.main(cache, tokens=10, quiet=True) < TOLERANCE[cache]
