"""A layer's run of the latent operators, each step against its own definition and both
forms of the attention against the layer's formula (latent_layer.py)."""
import pytest

import paged_varlen_attention_attn_gb300 as pa
from latent_layer import Layer, Package

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer():
    from paged_varlen_attention_attn_gb300 import _build
    _build.build()
    pa.load()
    s = Layer("cuda:0")
    s.run(Package())
    return s


@pytest.mark.parametrize("what", ["rows", "absorbed", "expanded", "formula"])
def test_a_layer(layer, what):
    getattr(layer, "check_" + what)()
