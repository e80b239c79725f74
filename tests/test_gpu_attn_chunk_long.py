"""Chunks over so many tokens that fp32 sums made one after the other would not hold them."""
import math

import numpy as np
import pytest

import attn_ref as R
from test_gpu_attn_chunk import P, _check, _i32, _pages, _run, _sees  # noqa: F401
from test_gpu_attn_decode import Paged, _dev, _host, _stored, _torch, _values

pytestmark = pytest.mark.gpu


def _alike(P, kv, D, n):  # noqa: F811
    """A cache of n tokens: keys of 0 but the first one's, values that are 64 to 95 64ths, and one 64th
    more for 10 of 32 tokens in a row."""
    import torch

    page = 256
    cache = P.KVCache.empty(n // page, 1, page, D, _torch(kv))
    cache.k.zero_()
    cache.k[0, 0, 0, 0] = 1
    codes = 64 + torch.arange(D, device="cuda") % 32 + (torch.arange(page, device="cuda")[:, None] % 32 < 10)
    if kv == "i8":
        cache.k_scale.fill_(1.0)
        cache.v.copy_(codes.to(torch.int8).expand(cache.v.shape))
        cache.v_scale.fill_(1 / 64)
    else:
        cache.v.copy_((codes / 64).bfloat16().expand(cache.v.shape))
    return cache, torch.arange(n // page, dtype=torch.int32, device="cuda")[None]


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_half_a_million_tokens_of_one_score(P, D, kv):  # noqa: F811
    """All keys but the first score 0 and have the weight w, a bf16 number.  With N tokens lse is
    ln(1 + (N - 1) w) - ln w.  A row's sum over 2^15 tokens is four of 2^13 terms: an addition rounds by
    2^-24 of the sum so far, half of the whole on average, so 2^12 2^-24 in all; sums of 16 such are joined
    with less than 2^-19.  The values of a dimension average a + 10/32 64ths: 5/8 of the bf16 step from a to
    a + 1/128, so an output is the latter unless it is off by 1/8 of that step, 2^-10.  The products of
    2^15 tokens, 16 at a time and truncated, are off by 2^11 / 2 units of 2^-23, 2^-13; with the sum's 2^-12, a row's
    unfinished 32 tokens and its first key (2^-13 / 64) and the joining under 2^-11.3 of values up to 1.5."""
    import torch

    n, nq, w = 1 << 19, 152 * 256, 0.69921875
    cache, table = _alike(P, kv, D, n)
    q = torch.zeros(nq, 1, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    lse = torch.empty(nq, 1, device="cuda")
    out = P.attn_chunk(q, cache, table, _i32([n]), _i32((0, nq)), scale=-math.log(w), lse=lse)
    P.device_check()
    seen = n - nq + 1 + torch.arange(nq, device="cuda", dtype=torch.float64)
    want = torch.log(1 + (seen - 1) * w) - math.log(w)
    off = (lse[:, 0].double() - want).abs()
    assert (off <= 2.0 ** -12 + 2.0 ** -20 * (2 + want)).all(), f"lse off by {off.max().item():.2e}"
    want = ((64 + torch.arange(D, device="cuda") % 32) / 64 + 1 / 128).bfloat16()
    wrong = (out[:, 0] != want).sum().item()
    assert wrong == 0, f"{wrong} of {out.numel()} outputs"


ROWS = (0, 1, 127, 128, 5000, 32639, 32767, 32768, 32769, 32895, 33023, 40000, 65535, 65536, 65791, 69000, 69999)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50000, 300)])
def test_a_long_prompt_in_one_chunk(P, D, kv, window, sinks):  # noqa: F811
    rng = np.random.default_rng(D + window)
    n = 70000
    s = Paged(P, rng, [n], 1, D, 256, kv)
    q = _values(rng, (n, 1, D), "bf16")
    out, lse = _run(P, s, q, (n,), window=window, sinks=sinks)
    k, v = _stored(s.k[0], kv), _stored(s.v[0], kv)
    rows = np.array(ROWS)
    ref = R.attend(q[rows, 0], k[:, 0], v[:, 0], D ** -0.5, _sees(rows, np.arange(n), window, sinks))
    R.check(out[rows, 0], lse[rows, 0], ref, True, True)


class Shared:
    """Sequences of the same pages."""

    def __init__(self, P, rng, n, B, D, kv):  # noqa: F811
        import torch

        one = Paged(P, rng, [n], 1, D, 256, kv)
        self.cache, self.kv, self.slots = one.cache, kv, one.slots
        self.table_d = one.table_d.expand(B, -1).contiguous()
        self.lens, self.k, self.v = [n] * B, one.k * B, one.v * B
        self.lens_d = torch.full((B,), n, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_few_tokens_of_many_long_sequences(P, D, kv):  # noqa: F811
    """More long contexts than CTAs: each goes over several of them."""
    rng = np.random.default_rng(D)
    n, B, nq, Hq = 66001, 310, 2, 3
    s = Shared(P, rng, n, B, D, kv)
    q = _values(rng, (B * nq, Hq, D), "bf16")
    for window, sinks in ((0, 0), (40000, 130)):
        out, lse = _run(P, s, q, [nq] * B, window=window, sinks=sinks)
        again = _run(P, s, q, [nq] * B, window=window, sinks=sinks)
        assert (out == again[0]).all() and (lse == again[1]).all()
        k, v = _stored(s.k[0], kv)[:, 0], _stored(s.v[0], kv)[:, 0]
        seen = _sees(n - nq + np.arange(nq), np.arange(n), window, sinks)
        for b in (0, 1, 77, 154, 309):
            for h in range(Hq):
                rows = b * nq + np.arange(nq)
                R.check(out[rows, h], lse[rows, h], R.attend(q[rows, h], k, v, D ** -0.5, seen), True, True, f"{b} {h}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_contexts_with_values_that_are_not_finite(P, D):  # noqa: F811
    """An infinite value among the first tokens, in the middle and at the end, which all rows see or the
    last one alone; and values whose sums overflow."""
    rng = np.random.default_rng(D + 5)
    n, B, nq, Hq = 66001, 310, 2, 2
    s = Shared(P, rng, n, B, D, "bf16")
    q = _values(rng, (B * nq, Hq, D), "bf16")
    seen = _sees(n - nq + np.arange(nq), np.arange(n), 0, 0)
    k, v = s.k[0][:, 0], s.v[0][:, 0]
    big = np.float32(3e38)
    for t, value in ((5, np.inf), (33000, -np.inf), (n - 1, np.inf), (n - 1, np.nan), (None, big)):
        keep = s.cache.v.clone()
        x = v.copy()
        if t is None:
            x[:, 1] = R.bf16(np.full(n, value))
            s.cache.v[..., 1] = float(value)
            k = R.bf16(k * np.linspace(0.1, 4, n)[:, None].astype(np.float32))       # maxima that grow
            import torch
            P.kv_write(s.cache, _dev(k[:, None], "bf16"), _dev(x[:, None], "bf16"), torch.from_numpy(s.slots).cuda())
        else:
            slot = int(s.slots[t])
            s.cache.v[slot // 256, 0, slot % 256, 1] = float(value)
        out, lse = _run(P, s, q, [nq] * B)
        for b in (0, 1, 154, 309):
            for h in range(Hq):
                rows = b * nq + np.arange(nq)
                o, l = out[rows, h], lse[rows, h]
                ref = R.attend(q[rows, h], k, x, D ** -0.5, seen)
                if t is None:
                    R.check(o, l, ref, True, True, f"{b} {h}")
                    continue
                hit = seen[:, t]
                assert not np.isfinite(o[hit, 1]).any()
                others = np.delete(np.arange(D), 1)
                R.check(o[:, others], l, (ref[0][:, others],) + ref[1:], True, True, f"{b} {h}")
                R.check(o[~hit], l[~hit], tuple(r[~hit] for r in ref), True, True, f"{b} {h}")
        s.cache.v.copy_(keep)
