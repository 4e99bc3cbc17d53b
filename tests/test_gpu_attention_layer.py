"""The attention layer's calls together, as examples/attention_layer.py runs
them, against the same layer in 64 bits.

Tolerance: two 8-bit roundings of activations stand in the way, each off by at
most 2^-4 and about 0.026 rms of the value; a projection keeps that relative
size (its terms are independent), and attention passes that of v on and turns
that of q and k into weights off by a few per cent: 0.1 over all."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from gated_delta_net_02_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    spec = importlib.util.spec_from_file_location(
        "attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("seqs,tokens", [(1, 1), (5, 1), (3, 4)])
def test_layer_against_64_bits(example, seqs, tokens):
    assert example.run(seqs, tokens, steps=3, prompt=30, check=True) < 0.1


def test_on_a_side_stream(example):
    with torch.cuda.stream(torch.cuda.Stream()):
        assert example.run(2, 2, steps=2, prompt=20, check=True, seed=5) < 0.1
