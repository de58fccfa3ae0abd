"""The served attention layer of examples/serve_attention_layer.py: projections, adapters, cache
and attention together, prompts and then tokens, against float64 over the decoded cache.

Bound: the attention's output and the layer's are f16 and the output projection holds Z in fp32, so
the error is that of two roundings of 2^-11 and of what the first does to the second's sum; 2^-8 of
the largest output leaves room for a factor of four between the largest and a typical value."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_served_layer(kind):
    spec = importlib.util.spec_from_file_location(
        "serve_attention_layer", os.path.join(ROOT, "examples", "serve_attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main(kind) <= 2.0 ** -8
