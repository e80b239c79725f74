"""Chunks over int8 whose queries and scales are near the ends of the range, though the
scores are not."""
import numpy as np
import pytest

import attn_ref as R
from test_gpu_attn_chunk import P, _i32, _pages, _sees  # noqa: F401
from test_gpu_attn_decode import _dev, _host, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 4)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("power", [126, 120, 115, -112, -119, -124])
def test_large_and_small_queries(P, D, power, window, sinks):  # noqa: F811
    """Queries of about 2^power, keys of codes and scales that bring the scores back to about 1: the sums of
    query times code pass 2^128, or none of their terms is a normal number."""
    import torch

    rng = np.random.default_rng(D)
    n, nq, Hq, page = 300, 40, 3, 16
    pages = -(-n // page)
    cache = P.KVCache.empty(pages, 1, page, D, torch.int8)
    codes = rng.integers(-127, 128, (2, pages, 1, page, D)).astype(np.int8)
    scales = np.full((2, pages, 1, page), 0.01, np.float32)
    scales[0] = np.float32(2.0) ** np.float32(-power - 6)
    for t, x in ((cache.k, codes[0]), (cache.v, codes[1]), (cache.k_scale, scales[0]), (cache.v_scale, scales[1])):
        t.copy_(torch.from_numpy(x).cuda())
    k, v = ((codes[i].astype(np.float64) * scales[i].astype(np.float64)[..., None])[:, 0].reshape(-1, D)[:n] for i in range(2))
    q = np.clip(_values(rng, (nq, Hq, D), "bf16"), -3, 3).astype(np.float64) * 2.0 ** (power - 1)
    q = R.bf16(q.astype(np.float32)).astype(np.float64)        # (small ones are rounded again)
    lse = torch.empty(nq, Hq, device="cuda")
    out = _host(P.attn_chunk(_dev(q.astype(np.float32), "bf16"), cache, _pages(np.arange(pages, dtype=np.int32)[None]), _i32([n]),
                             _i32((0, nq)), window=window, sinks=sinks, lse=lse))
    P.device_check()
    for h in range(Hq):
        seen = _sees(n - nq + np.arange(nq), np.arange(n), window, sinks)
        ref = R.attend(q[:, h], k, v, D ** -0.5, seen)
        assert np.abs(ref[1]).max() < 30
        R.check(out[:, h], _host(lse)[:, h], ref, True, True, f"head {h}")


@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** 109, 2.0 ** 111, 2.0 ** 125, 2.0 ** -125])
@pytest.mark.parametrize("D", [64, 256])
def test_large_and_small_softmax_scales(P, D, scale):  # noqa: F811
    """softmax_scale is any finite positive number."""
    import torch

    rng = np.random.default_rng(D + 2)
    n, nq, Hq, page = 200, 9, 2, 16
    pages = -(-n // page)
    cache = P.KVCache.empty(pages, 1, page, D, torch.int8)
    codes = rng.integers(-127, 128, (2, pages, 1, page, D)).astype(np.int8)
    scales = np.full((2, pages, 1, page), 0.01, np.float32)
    qs = 2.0 ** -60 if scale > 1 else 2.0 ** 60
    scales[0] = np.float32(1 / (scale * qs * 64 * D ** 0.5))       # q k scale is of the order of 1
    for t, x in ((cache.k, codes[0]), (cache.v, codes[1]), (cache.k_scale, scales[0]), (cache.v_scale, scales[1])):
        t.copy_(torch.from_numpy(x).cuda())
    k, v = ((codes[i].astype(np.float64) * scales[i].astype(np.float64)[..., None])[:, 0].reshape(-1, D)[:n] for i in range(2))
    q = R.bf16((_values(rng, (nq, Hq, D), "bf16") * np.float32(qs)).astype(np.float32))
    lse = torch.empty(nq, Hq, device="cuda")
    out = _host(P.attn_chunk(_dev(q, "bf16"), cache, _pages(np.arange(pages, dtype=np.int32)[None]), _i32([n]), _i32((0, nq)),
                             scale=scale, lse=lse))
    for h in range(Hq):
        ref = R.attend(q[:, h], k, v, float(np.float32(scale)), _sees(n - nq + np.arange(nq), np.arange(n), 0, 0))
        R.check(out[:, h], _host(lse)[:, h], ref, True, True, f"head {h}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_computed_again_keep_the_range(P, D):  # noqa: F811
    """Values whose sums overflow, under queries of 2^120: such rows are computed again from the codes."""
    import torch

    rng = np.random.default_rng(D + 3)
    n, nq, Hq, page = 260, 30, 2, 16
    pages = -(-n // page)
    cache = P.KVCache.empty(pages, 1, page, D, torch.int8)
    codes = rng.integers(-127, 128, (2, pages, 1, page, D)).astype(np.int8)
    codes[1] = np.abs(codes[1])
    scales = np.full((2, pages, 1, page), 2.0 ** -126, np.float32)
    scales[1] = np.float32(2.0 ** 120)                             # values up to 2^127
    for t, x in ((cache.k, codes[0]), (cache.v, codes[1]), (cache.k_scale, scales[0]), (cache.v_scale, scales[1])):
        t.copy_(torch.from_numpy(x).cuda())
    k, v = ((codes[i].astype(np.float64) * scales[i].astype(np.float64)[..., None])[:, 0].reshape(-1, D)[:n] for i in range(2))
    q = R.bf16((_values(rng, (nq, Hq, D), "bf16") * np.float32(2.0 ** 118)).astype(np.float32))
    out = _host(P.attn_chunk(_dev(q, "bf16"), cache, _pages(np.arange(pages, dtype=np.int32)[None]), _i32([n]), _i32((0, nq))))
    for h in range(Hq):
        ref = R.attend(q[:, h], k, v, D ** -0.5, _sees(n - nq + np.arange(nq), np.arange(n), 0, 0))
        R.check(out[:, h], None, ref, True, True, f"head {h}")
