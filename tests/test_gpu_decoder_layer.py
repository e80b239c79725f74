"""The decoder layer of examples/decoder_layer.py: prompts in chunks through
the paged int8 cache, then token by token, against the whole prompts at once.

The two runs see the same values but for roundings.  The prompt run holds
activations, keys, values and outputs of each product in bf16 (2^-9 relative
each), the served run reads keys and values of earlier tokens as int8
(half a step of max/127, about 2^-7 of a typical value) and computes the last
token in fp32.  Errors of independent values add as their squares: a relative
error of 2^-7 sqrt(2) from keys and values and 2^-9 from each of eight roundings
gives 1.25 %; twice that is allowed."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decoder_layer",
                                                  os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("hidden,q_heads,kv_heads,inner,tokens,chunk", [
    (1024, 8, 2, 2048, (150, 61), 64), (2048, 16, 8, 4096, (33, 90, 1), 200), (5120, 40, 8, 17408, (40, 17), 16)])
def test_served_and_whole_agree(example, hidden, q_heads, kv_heads, inner, tokens, chunk):
    last, full, x = example.run(hidden, q_heads, kv_heads, inner, tokens, chunk, steps=4)
    for a, b, c in zip(last, full, x):
        assert (a - b).norm() <= 0.025 * (b - c).norm()
