"""The C ABI of the paged cache and the attention over it, on the host:
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


def _cache(P, k=P16, v=P16, ks=P16, vs=P16, pages=4, page_tokens=16, kv_heads=2, head_dim=128, type=1):
    return P._KvCacheStruct(k, v, ks, vs, pages, page_tokens, kv_heads, head_dim, type)


BAD_CACHES = [(dict(k=None), 1), (dict(vs=None), 1), (dict(k=ODD), 3), (dict(ks=P16 + 2), 3),
              (dict(type=2), 4), (dict(head_dim=96), 5), (dict(head_dim=512), 5), (dict(head_dim=0), 2),
              (dict(pages=0), 2), (dict(page_tokens=0), 2), (dict(kv_heads=0), 2), (dict(pages=2 ** 27), 2),
              (dict(pages=2 ** 62), 2)]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_a_bad_cache_is_refused(P, bad, status):
    L = P.load()
    c = ctypes.byref(_cache(P, **bad))
    assert L.ptq_kv_write(c, P16, P16, 256, 256, P16, 3, P.PTQ_F32, None) == status
    assert L.ptq_kv_read(c, P16, 3, P16, P16, 256, 256, P.PTQ_F32, None) == status
    assert L.ptq_attn_decode(P16, 512, c, P16, 4, P16, P16, None, 2, 4, 0.1, P.PTQ_F32, P16, 1 << 40,
                             None) == status
    assert L.ptq_last_error()


def test_kv_rows(P):
    L = P.load()
    c = ctypes.byref(_cache(P))

    def both(k=P16, v=P16, ks=256, vs=256, slots=P16, T=3, dt=P.PTQ_F32, cache=c):
        a = L.ptq_kv_write(cache, k, v, ks, vs, slots, T, dt, None)
        assert a == L.ptq_kv_read(cache, slots, T, k, v, ks, vs, dt, None)
        return a

    assert both(cache=None) == 1
    assert both(k=None) == 1 and both(v=None) == 1 and both(slots=None) == 1
    assert both(k=ODD) == 3 and both(v=P16 + 8) == 3 and both(slots=P16 + 2) == 3
    assert both(ks=258) == 3 and both(vs=260, dt=P.PTQ_BF16) == 3
    assert both(ks=255) == 2 and both(vs=0) == 2 and both(T=-1) == 2 and both(T=2 ** 31) == 2
    assert both(ks=2 ** 62) == 2
    assert both(dt=7) == 4
    assert both(k=None, v=None, slots=None, T=0) == 0
    # a bf16 cache needs no scales
    assert both(cache=ctypes.byref(_cache(P, ks=None, vs=None, type=0)), T=0) == 0


def test_decode(P):
    L = P.load()
    c = ctypes.byref(_cache(P))
    need = P.attn_decode_workspace_bytes(2, 4, 2, 128, P.PTQ_F32)

    def call(q=P16, qs=512, cache=c, table=P16, width=4, lens=P16, out=P16, lse=None, B=2, Hq=4, scale=0.1,
             dt=P.PTQ_F32, ws=P16, wsb=1 << 40):
        return L.ptq_attn_decode(q, qs, cache, table, width, lens, out, lse, B, Hq, scale, dt, ws, wsb, None)

    assert call(cache=None) == 1
    for name in ("q", "table", "lens", "out"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: P16 + 2}) == 3, name
    assert call(q=ODD) == 3 and call(out=ODD) == 3 and call(lse=P16 + 2) == 3
    assert call(qs=514) == 3 and call(qs=511) == 2
    assert call(Hq=3) == 2 and call(Hq=0) == 2 and call(Hq=1) == 2
    assert call(B=-1) == 2 and call(width=-1) == 2 and call(width=2 ** 28) == 2 and call(B=2 ** 40) == 2
    for s in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=s) == 4
    assert call(dt=9) == 4
    if need:
        assert call(ws=None) == 6 and call(wsb=need - 1) == 6 and call(ws=ODD) == 3
    assert call(B=0, q=None, table=None, lens=None, out=None, ws=None, wsb=0) == 0
    for bad in ((-1, 4, 2, 128), (2, 5, 2, 128), (2, 4, 0, 128), (2, 4, 2, 96), (2 ** 40, 4, 2, 128)):
        assert P.attn_decode_workspace_bytes(*bad, P.PTQ_F32) == 0
    assert P.attn_decode_workspace_bytes(2, 4, 2, 128, 9) == 0


def test_prefill(P):
    L = P.load()
    need = P.attn_prefill_workspace_bytes(2, 10, 12, 4, 2, 128, P.PTQ_BF16)

    def call(q=P16, k=P16, v=P16, qs=512, ks=256, vs=256, cuq=P16, cuk=P16, out=P16, lse=None, B=2, Tq=10, Tk=12,
             Hq=4, Hkv=2, D=128, scale=0.1, flags=1, dt=P.PTQ_BF16, ws=P16, wsb=1 << 40):
        return L.ptq_attn_prefill(q, k, v, qs, ks, vs, cuq, cuk, out, lse, B, Tq, Tk, Hq, Hkv, D, scale, flags, dt,
                                  ws, wsb, None)

    for name in ("q", "k", "v", "cuq", "cuk", "out"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: P16 + 2}) == 3, name
    assert call(lse=P16 + 1) == 3
    assert call(qs=516) == 3 and call(ks=260) == 3 and call(vs=257) == 3
    assert call(qs=511) == 2 and call(ks=255) == 2 and call(vs=128) == 2
    assert call(Hq=5) == 2 and call(Hkv=0) == 2 and call(Tq=-1) == 2 and call(Tk=2 ** 31) == 2 and call(B=-1) == 2
    assert call(D=96, qs=512) == 5 and call(D=320, qs=2048, ks=1024, vs=1024) == 5
    assert call(dt=P.PTQ_F32) == 5
    assert b"f32" in L.ptq_last_error()
    assert call(dt=9) == 4 and call(flags=2) == 4
    for s in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=s) == 4
    if need:
        assert call(ws=None) == 6 and call(wsb=need - 1) == 6 and call(ws=ODD) == 3
    assert call(B=0, q=None, k=None, v=None, cuq=None, cuk=None, out=None, ws=None, wsb=0) == 0
    assert call(Tq=0, q=None, out=None, ws=None, wsb=0) == 0
    for bad in ((-1, 10, 12, 4, 2, 128), (2, -1, 12, 4, 2, 128), (2, 10, 12, 5, 2, 128), (2, 10, 12, 4, 2, 100)):
        assert P.attn_prefill_workspace_bytes(*bad, P.PTQ_BF16) == 0
    assert P.attn_prefill_workspace_bytes(2, 10, 12, 4, 2, 128, P.PTQ_F32) == 0


def test_binding_checks(P):
    import torch

    z = torch.zeros(2, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        P.KVCache(z, z)
    with pytest.raises(ValueError, match="of one type"):
        P.KVCache(z, z[:1])
    with pytest.raises(ValueError, match="scale"):
        P.KVCache(z.to(torch.int8), z.to(torch.int8))
    with pytest.raises(TypeError, match="bfloat16 or int8"):
        P.KVCache(z.float(), z.float())
    with pytest.raises(ValueError, match="no scales"):
        P.KVCache(z, z, z, z)


def test_more_sequences_than_can_be_counted_are_refused(P):
    L = P.load()
    c = ctypes.byref(_cache(P, kv_heads=1, head_dim=64))
    assert L.ptq_attn_decode(P16, 64, c, P16, 4, P16, P16, None, 2 ** 30, 1, 0.1, P.PTQ_BF16, P16, 1 << 40,
                             None) == 2
    assert L.ptq_attn_prefill(P16, P16, P16, 64, 64, 64, P16, P16, P16, None, 2 ** 30, 8, 8, 1, 1, 64, 0.1, 0,
                              P.PTQ_BF16, P16, 1 << 40, None) == 2
    assert L.ptq_attn_decode_workspace_bytes(2 ** 30, 1, 1, 64, P.PTQ_BF16) == 0
    assert L.ptq_attn_prefill_workspace_bytes(2 ** 30, 8, 8, 1, 1, 64, P.PTQ_BF16) == 0
