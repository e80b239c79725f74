"""The edges of the paged cache and the attention operators: rows of the
smallest subnormals, value scales that differ by orders of magnitude."""
import numpy as np
import pytest

import attn_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import ternary_weight_ptq1_gb300 as P

    P.load()
    return P


def _host(t):
    return t.double().cpu().numpy()


# ---- the cache -------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128, 256])
def test_codes_of_subnormal_rows_stay_in_range(P, D):
    """Under a maximum of some 2^-135 the scale max / 127 is a subnormal of few
    bits, and the quotients pass 127: the codes stop there."""
    import torch

    unit = 2.0 ** -149
    tops = [1, 63, 64, 127, 128, 190, 191, 255, 318, 5000, 70001, 2 ** 20 + 1, 2 ** 23 - 1, 2 ** 23, 2 ** 24]
    rng = np.random.default_rng(D)
    x = np.zeros((2 * len(tops), 1, D), np.float32)
    for i, top in enumerate(tops):
        x[2 * i:2 * i + 2, 0] = rng.integers(-top, top + 1, D) * unit
        x[2 * i, 0, 5], x[2 * i + 1, 0, D - 1] = top * unit, -top * unit
    xd = torch.from_numpy(x).cuda()
    cache = P.KVCache.empty(len(x), 1, 1, D, torch.int8)
    slots = torch.arange(len(x), dtype=torch.int32, device="cuda")
    P.kv_write(cache, xd, -xd, slots)
    s = np.abs(x).max(-1) / np.float32(127)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s[..., None] > 0, np.clip(np.rint(x / s[..., None]), -127, 127), 0).astype(np.int8)
    assert (np.abs(c) == 127).any() and (s == 0).any()
    np.testing.assert_array_equal(cache.k_scale.cpu().numpy()[:, 0], s)
    np.testing.assert_array_equal(cache.k.cpu().numpy()[:, 0], c)
    np.testing.assert_array_equal(cache.v.cpu().numpy()[:, 0], -c)
    k, v = P.kv_read(cache, slots, dtype=torch.float32)
    np.testing.assert_array_equal(k.cpu().numpy(), c * s[..., None])
    np.testing.assert_array_equal(v.cpu().numpy(), -c * s[..., None])
