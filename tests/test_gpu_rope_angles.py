"""The angles that heads are turned by, against exact ones at any position."""
import math

import numpy as np
import pytest

import attn_ref as A
from test_gpu_rope import P, _dev, _host  # noqa: F401

pytestmark = pytest.mark.gpu

BITS = 256


def _turns_of_one():
    """1 / (2 pi) times 2^BITS, by Machin's formula in integers."""
    one = 1 << (2 * BITS)

    def arctan_of_one_over(n):
        term = total = one // n
        k = 1
        while term:
            term //= n * n
            total += (-1) ** k * (term // (2 * k + 1))
            k += 1
        return total
    pi = 4 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239))       # times 2^(2 BITS)
    return (one << BITS) // (2 * pi)


def _angles(pos, f):
    """pos times f without its whole turns, in radians of (-pi, pi]."""
    m, e = math.frexp(float(f))
    m, e = int(m * 2 ** 24), e - 24
    t = pos * m * _angles.turn                                             # turns, times 2^(BITS - e)
    t = t << e if e >= 0 else t >> -e
    t &= (1 << BITS) - 1
    if t >> (BITS - 1):
        t -= 1 << BITS
    return t / (1 << BITS) * (2 * math.pi)


_angles.turn = _turns_of_one()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D", [64, 256])
def test_angles_are_right_to_a_part_of_two_to_the_27_of_a_turn(P, D, interleaved):  # noqa: F811
    """(1, 0) turned by t is (cos t, sin t) with no other rounding: products with 1 and 0 are exact.  An angle is
    rounded to fp32 within an eighth of a turn either way, to 2^-28 of a turn, and in its integers to 2^-31: under
    2^-27 of a turn together; sines and cosines are within 2 units in their last place."""
    import torch

    rng = np.random.default_rng(D)
    half, T = D // 2, 400
    inv = np.concatenate([1e4 ** (-np.arange(half - 8) / (half - 8)), rng.uniform(-4, 4, 4),
                          [2.0 ** 32, 123456.789, -3e9, 2.0 ** -20]]).astype(np.float32)
    pos = np.concatenate([rng.integers(0, 4096, T // 4), rng.integers(0, 10 ** 6, T // 4),
                          rng.integers(-2 ** 31, 2 ** 31, T // 2 - 2), [2 ** 31 - 1, -2 ** 31]]).astype(np.int32)
    x = np.zeros((T, 1, D), np.float32)
    first, second = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), half + np.arange(half))
    x[..., first] = 1.0
    y, _ = P.qk_rope(P.Rope(_dev(inv), interleaved=interleaved), _dev(x), _dev(x), _dev(pos))
    torch.cuda.synchronize()
    y = _host(y)[:, 0]
    t = np.array([[_angles(int(p), f) for f in inv] for p in pos])
    off, unit = 2 * np.pi * 2.0 ** -27, 2.0 ** -23
    c, s = np.cos(t), np.sin(t)
    ec, es = np.abs(y[:, first] - c), np.abs(y[:, second] - s)
    worst = max((ec - off * np.abs(s) - unit * np.abs(c)).max(), (es - off * np.abs(c) - unit * np.abs(s)).max())
    assert worst <= off ** 2, f"{worst:.2e}"


def test_quarters_of_a_turn_are_exact_in_bf16_as_well(P):  # noqa: F811
    """Angles on every side of each eighth of a turn."""
    D, half = 64, 32
    inv = np.full(half, np.float32(math.pi / 4))
    inv[1::2] = np.nextafter(inv[0], np.float32(0))
    pos = np.concatenate([np.arange(-40, 40), 2 ** np.arange(6, 31), -2 ** np.arange(6, 31)]).astype(np.int32)
    x = A.bf16(np.random.default_rng(3).standard_normal((len(pos), 1, D)).astype(np.float32))
    for act in ("f32", "bf16"):
        y, _ = P.qk_rope(P.Rope(_dev(inv)), _dev(x, act), _dev(x, act), _dev(pos))
        t = np.array([[_angles(int(p), f) for f in inv] for p in pos])
        a, b = x[:, 0, :half].astype(np.float64), x[:, 0, half:].astype(np.float64)
        want = np.concatenate([a * np.cos(t) - b * np.sin(t), b * np.cos(t) + a * np.sin(t)], -1)
        size = np.tile(np.abs(a) + np.abs(b), 2)
        bound = 2 * np.pi * 2.0 ** -27 * size + 6 * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(want) if act == "bf16" else 0)
        assert (np.abs(_host(y)[:, 0] - want) <= bound).all()
