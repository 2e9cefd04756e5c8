"""The example that runs the 4-bit operators together: every layer's output against fp64."""
import importlib.util
import os

import pytest

from conv_activation_epilogue_gb300 import build, mmact

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    build.build()
    mmact.load()
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "mixture_block.py")
    spec = importlib.util.spec_from_file_location("mixture_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("tokens", [1, 9, 64, 131])
def test_each_layer_is_its_formula(example, tokens):
    block = example.build(D=520, H=1024, I=392, E=12, top=3, max_tokens=131, seed=tokens)
    # one rounding to bf16, 2^-9 of a value at most, and the fp32 sums, which are far below it
    assert all(e <= 2.0 ** -8 for e in example.errors(block, tokens))


def test_the_block_runs_as_a_graph(example):
    block = example.build(D=256, H=512, I=200, E=8, top=2, max_tokens=4)
    assert example.time_graph(block, 4, 3) > 0
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
