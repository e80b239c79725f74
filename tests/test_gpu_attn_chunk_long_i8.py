"""Chunks over long int8 contexts whose scales or pages are not sound, and over workspaces that hold anything."""
import numpy as np
import pytest

import attn_ref as R
from test_gpu_attn_chunk import P, _i32, _run, _sees  # noqa: F401
from test_gpu_attn_chunk_long import Shared
from test_gpu_attn_decode import _dev, _stored, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("what", ["v_scale", "k_scale", "page"])
def test_rows_that_see_it_are_nan_and_no_others(P, D, what):  # noqa: F811
    rng = np.random.default_rng(D)
    n, B, nq, Hq = 66001, 310, 2, 2
    s = Shared(P, rng, n, B, D, "i8")
    q = _values(rng, (B * nq, Hq, D), "bf16")
    k, v = _stored(s.k[0], "i8")[:, 0], _stored(s.v[0], "i8")[:, 0]
    for window, sinks in ((0, 0), (40000, 130)):
        seen = _sees(n - nq + np.arange(nq), np.arange(n), window, sinks)
        refs = {}
        for t in (5, 20000, 33000, n - 1):
            if what == "page":
                keep = s.table_d.clone()
                s.table_d[:, t // 256] = -1 if t != n - 1 else 10 ** 8
                hit = seen[:, t // 256 * 256:min(n, t // 256 * 256 + 256)].any(1)
            else:
                scale = getattr(s.cache, what)
                keep = scale.clone()
                slot = int(s.slots[t])
                scale[slot // 256, 0, slot % 256] = float("nan")
                hit = seen[:, t]
            out, lse = _run(P, s, q, [nq] * B, window=window, sinks=sinks)
            for b in (0, 1, 154, 309):
                rows = b * nq + np.arange(nq)
                assert np.isnan(out[rows[hit]]).all()
                for h in range(Hq):
                    ref = refs.setdefault((b, h), R.attend(q[rows, h], k, v, D ** -0.5, seen))
                    R.check(out[rows[~hit], h], lse[rows[~hit], h], tuple(r[~hit] for r in ref), True, True, f"{t} {b} {h}")
                    if what == "v_scale":
                        assert np.allclose(lse[rows, h], ref[1], 0, 1e-4)
                    else:
                        assert np.isnan(lse[rows[hit], h]).all()
            (s.table_d if what == "page" else scale).copy_(keep)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("D", [64, 256])
def test_workspaces_may_hold_anything(P, D, kv):  # noqa: F811
    """Sums that pass through the workspace are written before they are read, as the call repeats over any contents."""
    import torch

    rng = np.random.default_rng(D + 9)
    n, B, nq, Hq = 66001, 310, 2, 3
    s = Shared(P, rng, n, B, D, kv)
    q = _dev(_values(rng, (B * nq, Hq, D), "bf16"), "bf16")
    cu = _i32(range(0, B * nq + 1, nq))
    need = P.attn_chunk_workspace_bytes(B, B * nq, Hq, 1, D, P.PTQ_BF16)
    got = []
    for fill in (0, 255, 127):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        ws[need:] = 170
        got.append(P.attn_chunk(q, s.cache, s.table_d, s.lens_d, cu, workspace=ws[:need]))
        assert (ws[need:] == 170).all() and torch.isfinite(got[-1]).all()
    P.device_check()
    assert all(torch.equal(g, got[0]) for g in got)
