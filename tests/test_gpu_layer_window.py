"""The decoder layer of examples/decoder_layer.py under a sliding window: its
prompts in chunks and then token by token, against the whole prompts at once,
both through the cache.  The two see the same int8 keys and values; the
activations of the prompt run are rounded to bf16 (2^-9 relative, eight roundings),
the served run's last token is fp32: the layer's 1.25 % of test_gpu_decoder_layer
holds, twice that is allowed."""
import pytest

from test_gpu_decoder_layer import example  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hidden,q_heads,kv_heads,inner,tokens,chunk,window", [
    (1024, 8, 2, 2048, (150, 61), 64, 40), (2048, 16, 8, 4096, (333, 90, 1), 200, 128)])
def test_served_and_whole_agree_under_a_window(example, hidden, q_heads, kv_heads, inner, tokens, chunk, window):  # noqa: F811
    last, full, x = example.run(hidden, q_heads, kv_heads, inner, tokens, chunk, steps=4, window=window)
    for a, b, c in zip(last, full, x):
        assert (a - b).norm() <= 0.025 * (b - c).norm()


def test_a_window_changes_the_outputs(example):  # noqa: F811
    _, near, _ = example.run(1024, 8, 2, 2048, (150,), 64, steps=1, window=8)
    _, far, _ = example.run(1024, 8, 2, 2048, (150,), 64, steps=1)
    assert (near - far).abs().max() > 0
