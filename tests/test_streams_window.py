"""attn_decode refuses numbers of first tokens with and without a window, as the C call does."""
import pytest

from test_abi_rope import P, _window  # noqa: F401
from test_streams import world  # noqa: F401
from test_streams_rope import _things


@pytest.mark.parametrize("sinks", [-1, 2 ** 31, 2 ** 40])
@pytest.mark.parametrize("window", [0, 5])
def test_the_library_refuses_it(P, window, sinks):  # noqa: F811
    assert _window(P, window=window, sinks=sinks) == 4


@pytest.mark.parametrize("sinks", [-1, 2 ** 31, 2 ** 40])
@pytest.mark.parametrize("window", [0, 5])
def test_and_is_asked(world, window, sinks):  # noqa: F811
    P, cache, _, t = _things(world)
    P.attn_decode(t["q"], cache, t["table4"], t["lens4"], window=window, sinks=sinks)
    (name, args), = world.calls
    assert name == "ptq_attn_decode_window" and args[11:13] == (window, sinks)


def test_without_a_window_first_tokens_count_for_nothing(world):  # noqa: F811
    P, cache, _, t = _things(world)
    for sinks in (0, 1, 2 ** 31 - 1):
        P.attn_decode(t["q"], cache, t["table4"], t["lens4"], sinks=sinks)
    assert [n for n, _ in world.calls] == ["ptq_attn_decode"] * 3
