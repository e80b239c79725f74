"""Chunks whose keys go over two sums, one of them far below the other: what is not
finite there stays so."""
import numpy as np
import pytest

import attn_ref as R
from test_gpu_attn_chunk import P, _run, _sees  # noqa: F401
from test_gpu_attn_decode import Paged, _dev, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq", [(64, 7), (128, 5), (256, 6)])
@pytest.mark.parametrize("n,gap", [(256, 100.0), (256, 128.0), (640, 128.0), (1000, 400.0)])
def test_a_seen_value_counts_however_low_its_score(P, D, Hq, n, gap):  # noqa: F811
    """Scores of one tile of keys are so far below the others' that their weights are 0 in fp32.  An
    infinite value there is seen all the same: 0 times it is not finite, whichever sum it went to."""
    import torch

    rng = np.random.default_rng(n)
    nq = 4
    s = Paged(P, rng, [n], 1, D, 16, "bf16")
    q = _values(rng, (nq, Hq, D), "bf16")
    q[..., 0] = 4.0
    for low in range(-(-n // 128)):
        s.k[0][..., 0] = 0.0
        s.k[0][low * 128:low * 128 + 128, :, 0] = -gap / 4
        v = s.v[0].copy()
        t = min(low * 128 + 5, n - nq)                         # every query sees it
        v[t, 0, 3] = np.inf
        P.kv_write(s.cache, _dev(s.k[0], "bf16"), _dev(v, "bf16"), torch.from_numpy(s.slots).cuda())
        out, lse = _run(P, s, q, (nq,), scale=1.0)
        others = np.delete(np.arange(D), 3)
        seen = _sees(n - nq + np.arange(nq), np.arange(n), 0, 0)
        for h in range(Hq):
            ref = R.attend(q[:, h], s.k[0][:, 0], s.v[0][:, 0], 1.0, seen)
            R.check(out[:, h][:, others], lse[:, h], (ref[0][:, others],) + ref[1:], True, True, f"tile {low} head {h}")
        assert not np.isfinite(out[..., 3]).any(), f"tile {low}"
