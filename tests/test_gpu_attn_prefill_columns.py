"""Prompts over values of which some are not finite and others so large that their weighted sums
overflow: each dimension of an output goes by its own values."""
import numpy as np
import pytest

import attn_ref as R
from test_gpu_attn_prefill import P, _cu, _host  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,G", [(64, 7), (128, 5), (256, 6), (128, 1)])
def test_an_infinite_value_leaves_other_dimensions(P, D, G, causal):  # noqa: F811
    """Weights may be 2^8 times the largest key's while they are summed, and the sums of values near 1e36
    then overflow (147 x 132 x 1e36); relative to the largest key (132 x 1e36) they do not.  An infinite value
    that a row sees in one dimension says nothing of the others."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(D)
    n, nq = 260, 60
    q = torch.zeros(nq, G, D, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(n, 1, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0], k[128:, 0, 0] = 1.0, 5.0     # scores of 0, then of 5 (7.2 in units of log2)
    v = (torch.rand(n, 1, D, device="cuda", generator=gen) + 0.5).mul(1e36).bfloat16()
    column, others = D - 1, np.arange(D - 1)
    for t in (None, 5, 150, 230):
        x = v.clone()
        if t is not None:
            x[t, 0, column] = float("inf")
        out = _host(P.attn_prefill(q, k, x, _cu([nq]), _cu([n]), causal=causal, scale=1.0))
        P.device_check()
        for i in (0, 1, nq // 2, nq - 1):
            m = n - nq + i + 1 if causal else n
            ref = R.attend(_host(q[i]), _host(k[:m, 0]), _host(v[:m, 0]), 1.0)
            sees = t is not None and t < m
            R.check(out[i][:, others], None, (ref[0][:, others],) + ref[1:], True, True, f"token {t} row {i}")
            assert np.isfinite(out[i][:, column]).all() == (not sees)
