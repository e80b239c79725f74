"""Chunks over values of which some are not finite and others so large that their weighted
sums overflow: each dimension of an output goes by its own values."""
import numpy as np
import pytest

import attn_ref as R
from test_gpu_attn_chunk import P, _run, _sees  # noqa: F401
from test_gpu_attn_decode import Paged, _dev, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(0, 0), (120, 8)])
@pytest.mark.parametrize("D,Hq", [(64, 7), (128, 5), (256, 6)])
def test_an_infinite_value_leaves_other_dimensions(P, D, Hq, window, sinks):  # noqa: F811
    """Values of 3e38 of one sign a dimension have a mean, though weights of up to 2^8 make their sum
    overflow; an infinite value that a row sees in one dimension says nothing of the others."""
    import torch

    rng = np.random.default_rng(41)
    n, nq = 500, 200
    s = Paged(P, rng, [n], 1, D, 16, "bf16")
    s.v[0] = R.bf16(np.sign(s.v[0][:1]) * np.float32(3e38) * np.ones_like(s.v[0]))
    s.k[0] = R.bf16(s.k[0] * np.linspace(0.1, 6, n)[:, None, None].astype(np.float32))     # maxima that grow
    q = _values(rng, (nq, Hq, D), "bf16")
    column, others = D - 1, np.arange(D - 1)
    for t in (5, 250, 380, n - 1):
        v = s.v[0].copy()
        v[t, 0, column] = np.inf
        P.kv_write(s.cache, _dev(s.k[0], "bf16"), _dev(v, "bf16"), torch.from_numpy(s.slots).cuda())
        out, lse = _run(P, s, q, (nq,), window=window, sinks=sinks)
        seen = _sees(n - nq + np.arange(nq), np.arange(n), window, sinks)
        hit = seen[:, t]
        assert not np.isfinite(out[hit][..., column]).any(), f"token {t}"
        use = np.unique(np.r_[0, nq - 1, np.flatnonzero(hit)[:1], np.flatnonzero(~hit)[:1], rng.permutation(nq)[:4]])
        for h in range(Hq):
            ref = R.attend(q[use, h], s.k[0][:, 0], s.v[0][:, 0], D ** -0.5, seen[use])
            R.check(out[use, h][:, others], lse[use, h], (ref[0][:, others],) + ref[1:], True, True, f"token {t} head {h}")
            free = ~hit[use]
            part = tuple(r[free] for r in ref)
            R.check(out[use[free], h], lse[use[free], h], part, True, True, f"token {t} head {h}, rows that do not see it")
