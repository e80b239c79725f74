"""The C ABI of head norms, rotation, appending, chunks and windows, on the host:
every refusal comes before any launch.  No call here touches a GPU."""
import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def P():
    import ternary_weight_ptq1_gb300 as P

    P._build.build()
    P.load()
    return P


P16, ODD = 16 * 1024, 16 * 1024 + 4      # never dereferenced: every call here is refused


def _cache(P, **bad):
    f = dict(k=P16, v=P16, k_scale=P16, v_scale=P16, pages=4, page_tokens=16, kv_heads=2, head_dim=128, type=1)
    f.update(bad)
    return P._KvCacheStruct(**f)


def _rope(P, **bad):
    f = dict(inv_freq=P16, axis=None, pos=P16, pos_stride=3, axes=1, rotary_dim=128, interleaved=0, q_gain=P16,
             k_gain=P16, eps=1e-6)
    f.update(bad)
    return P._RopeStruct(**f)


def _qk(P, rope=None, q=P16, k=P16, qs=512, ks=256, qo=P16, ko=P16, qos=512, kos=256, T=3, Hq=4, Hkv=2, D=128, dt=0):
    r = ctypes.byref(_rope(P, **(rope or {})))
    return P.load().ptq_qk_rope(r, q, k, qs, ks, qo, ko, qos, kos, T, Hq, Hkv, D, dt, None)


def _append(P, rope=None, cache=None, q=P16, k=P16, v=P16, qs=512, ks=256, vs=256, slots=P16, qo=P16, qos=512, T=3,
            Hq=4, dt=0):
    return P.load().ptq_kv_append(ctypes.byref(_cache(P, **(cache or {}))), ctypes.byref(_rope(P, **(rope or {}))), q, k,
                                  v, qs, ks, vs, slots, qo, qos, T, Hq, dt, None)


BAD_ROPES = [(dict(inv_freq=None), 1), (dict(pos=None), 1), (dict(rotary_dim=-8), 2), (dict(rotary_dim=132), 2),
             (dict(rotary_dim=136), 2), (dict(rotary_dim=4), 2), (dict(axes=0), 2), (dict(axes=128, pos_stride=9), 2),
             (dict(axes=2, pos_stride=2), 2), (dict(axes=3, pos_stride=-1), 2), (dict(axes=3, pos_stride=2 ** 62), 2),
             (dict(eps=0.0), 4), (dict(eps=-1.0), 4), (dict(eps=math.inf), 4), (dict(eps=math.nan), 4),
             (dict(q_gain=ODD), 3), (dict(k_gain=P16 + 8), 3), (dict(inv_freq=P16 + 2), 3), (dict(pos=P16 + 1), 3)]


@pytest.mark.parametrize("bad,status", BAD_ROPES)
def test_a_bad_rope_is_refused(P, bad, status):
    assert _qk(P, rope=bad) == status and P.load().ptq_last_error()
    assert _append(P, rope=bad) == status and P.load().ptq_last_error()


def test_what_a_rope_does_not_use_is_not_asked_for(P):
    # no rotation: no frequencies and positions; no gains: no eps; nothing to do: no pointers
    none = dict(rotary_dim=0, inv_freq=None, pos=None, axes=0, q_gain=None, k_gain=None, eps=0.0)
    assert _qk(P, rope=none, T=0, q=None, k=None, qo=None, ko=None) == 0
    assert _append(P, rope=none, T=0, q=None, k=None, v=None, slots=None, qo=None) == 0
    assert _append(P, rope=dict(pos=None, inv_freq=None), T=0) == 0
    assert P.load().ptq_qk_rope(None, P16, P16, 512, 256, P16, P16, 512, 256, 3, 4, 2, 128, 0, None) == 1
    assert P.load().ptq_kv_append(ctypes.byref(_cache(P)), None, P16, P16, P16, 512, 256, 256, P16, P16, 512, 3, 4, 0,
                                  None) == 1


def test_qk_rope(P):
    for name in ("q", "k", "qo", "ko"):
        assert _qk(P, **{name: None}) == 1, name
        assert _qk(P, **{name: ODD}) == 3, name
    for name, low in (("qs", 511), ("ks", 255), ("qos", 500), ("kos", 0)):
        assert _qk(P, **{name: low}) == 2, name
        assert _qk(P, **{name: 2 ** 62}) == 2, name
        assert _qk(P, **{name: 514}) == 3, name
    assert _qk(P, T=-1) == 2 and _qk(P, T=2 ** 31) == 2
    assert _qk(P, Hq=-1) == 2 and _qk(P, Hq=0, Hkv=0) == 2 and _qk(P, Hq=2 ** 21, qs=2 ** 30, qos=2 ** 30) == 2
    assert _qk(P, D=96) == 5 and _qk(P, D=512) == 5 and _qk(P, D=0) == 2
    assert _qk(P, dt=7) == 4
    # a side without heads needs no tensor: the other's fault is found
    assert _qk(P, Hq=0, q=None, qo=None, ko=None) == 1 and _qk(P, Hkv=0, k=None, ko=None, qo=ODD) == 3


def test_kv_append(P):
    for name in ("k", "v", "slots", "q", "qo"):
        assert _append(P, **{name: None}) == 1, name
        assert _append(P, **{name: P16 + 2}) == 3, name
    assert _append(P, cache=dict(head_dim=96)) == 5 and _append(P, cache=dict(k=None)) == 1
    assert _append(P, cache=dict(type=3)) == 4 and _append(P, cache=dict(k_scale=None)) == 1
    assert _append(P, ks=255) == 2 and _append(P, vs=258) == 3 and _append(P, qs=100) == 2 and _append(P, qos=100) == 2
    assert _append(P, T=-1) == 2 and _append(P, T=2 ** 31) == 2 and _append(P, Hq=-1) == 2
    assert _append(P, dt=9) == 4
    assert _append(P, Hq=0, q=None, qo=None, qs=0, qos=0, slots=None) == 1     # no queries: their tensors are not looked at


def _chunk(P, q=P16, qs=512, cache=None, table=P16, width=4, lens=P16, cu=P16, out=P16, lse=None, B=2, Tq=10, Hq=4,
           scale=0.1, window=0, sinks=0, dt=1, ws=P16, wsb=1 << 40):
    return P.load().ptq_attn_chunk(q, qs, ctypes.byref(_cache(P, **(cache or {}))), table, width, lens, cu, out, lse, B,
                                   Tq, Hq, scale, window, sinks, dt, ws, wsb, None)


def _window(P, q=P16, qs=512, cache=None, table=P16, width=4, lens=P16, out=P16, lse=None, B=2, Hq=4, scale=0.1,
            window=8, sinks=0, dt=0, ws=P16, wsb=1 << 40):
    return P.load().ptq_attn_decode_window(q, qs, ctypes.byref(_cache(P, **(cache or {}))), table, width, lens, out, lse,
                                           B, Hq, scale, window, sinks, dt, ws, wsb, None)


@pytest.mark.parametrize("call", [_chunk, _window])
def test_chunk_and_window(P, call):
    for name in ("q", "table", "lens", "out") + (("cu",) if call is _chunk else ()):
        assert call(P, **{name: None}) == 1, name
        assert call(P, **{name: P16 + 2}) == 3, name
    assert call(P, q=ODD) == 3 and call(P, out=ODD) == 3 and call(P, lse=P16 + 2) == 3
    assert call(P, qs=514) == 3
    assert call(P, qs=511) == 2 and call(P, Hq=3) == 2 and call(P, Hq=0) == 2 and call(P, B=-1) == 2
    assert call(P, width=-1) == 2 and call(P, width=2 ** 28) == 2 and call(P, B=2 ** 40) == 2
    for s in (0.0, -1.0, math.inf, math.nan):
        assert call(P, scale=s) == 4
    for w in (-1, 2 ** 31, 2 ** 40):
        assert call(P, window=w) == 4 and call(P, sinks=w) == 4
    assert call(P, dt=9) == 4
    assert call(P, cache=dict(head_dim=96)) == 5 and call(P, cache=dict(v=None)) == 1
    assert call(P, B=0, q=None, table=None, lens=None, out=None, ws=None, wsb=0) == 0


def test_chunk_alone(P):
    need = P.attn_chunk_workspace_bytes(2, 10, 4, 2, 128, P.PTQ_BF16)
    if need:
        assert _chunk(P, ws=None) == 6 and _chunk(P, wsb=need - 1) == 6 and _chunk(P, ws=ODD) == 3
    assert _chunk(P, dt=0) == 5 and b"f32" in P.load().ptq_last_error()
    big = dict(pages=2 ** 20, page_tokens=256, kv_heads=1, head_dim=64)
    most = dict(cache=big, qs=256, Hq=4)
    assert _chunk(P, width=2 ** 19 + 1, **most) == 5 and _chunk(P, width=2 ** 19 + 1, window=2 ** 27, sinks=1, **most) == 5
    assert _chunk(P, width=2 ** 19 + 1, window=2 ** 27, ws=None, **most) == 6       # (as far as the workspace)
    assert _chunk(P, Tq=-1) == 2 and _chunk(P, Tq=2 ** 31) == 2 and _chunk(P, B=2 ** 26) == 2
    assert _chunk(P, Tq=0, q=None, out=None, ws=None, wsb=0) == 0
    for bad in ((-1, 10, 4, 2, 128), (2, -1, 4, 2, 128), (2, 10, 5, 2, 128), (2, 10, 4, 2, 100), (2 ** 26, 10, 4, 2, 128)):
        assert P.attn_chunk_workspace_bytes(*bad, P.PTQ_BF16) == 0
    assert P.attn_chunk_workspace_bytes(2, 10, 4, 2, 128, P.PTQ_F32) == 0


def test_binding_checks(P):
    import torch

    f = torch.ones(32)
    with pytest.raises(TypeError, match="CUDA"):
        P.Rope(f)
    with pytest.raises(ValueError, match="axis"):
        P.Rope(f, axis=torch.zeros(31, dtype=torch.int8))
    with pytest.raises(ValueError, match="head_dim"):
        P.Rope(f, q_gain=torch.ones(2, 64))
