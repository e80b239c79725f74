"""Chunks over the paged cache where they can go wrong: shapes, alignments, contents
of the cache that kv_write does not make, many sequences without queries, graphs,
and norms, rotation, appending and attention in a row."""
import numpy as np
import pytest

import attn_ref as R
import rope_ref
from test_gpu_attn_chunk import P, _check, _i32, _pages, _run, _sees  # noqa: F401
from test_gpu_attn_decode import Paged, _dev, _host, _torch, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("Hq,Hkv", [(13, 1), (130, 1), (64, 1), (128, 1), (9, 9), (26, 2), (257, 1)])
def test_numbers_of_heads(P, Hq, Hkv, kv):  # noqa: F811
    rng = np.random.default_rng(Hq)
    lens, nq = [150, 3], (11, 2)
    s = Paged(P, rng, lens, Hkv, 64, 16, kv)
    q = _values(rng, (13, Hq, 64), "bf16")
    out, lse = _run(P, s, q, nq)
    _check(s, q, nq, out, lse, rows=3, rng=rng)


def test_no_tokens_and_no_table(P):  # noqa: F811
    import torch

    cache = P.KVCache.empty(1, 1, 16, 64, torch.bfloat16)
    q = torch.randn(5, 2, 64, device="cuda").bfloat16()
    lse = torch.zeros(5, 2, device="cuda")
    for width in (0, 1):
        out = P.attn_chunk(q, cache, torch.full((2, width), -1, dtype=torch.int32, device="cuda"),
                           _i32((0 if width else 9, -3)), _i32((0, 2, 5)), lse=lse)
        assert (out == 0).all() and torch.isneginf(lse).all()
    assert P.attn_chunk(q[:0], cache, torch.zeros((2, 1), dtype=torch.int32, device="cuda"), _i32((4, 4)),
                        _i32((0, 0, 0))).shape == (0, 2, 64)
    P.device_check()


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_many_sequences_without_queries(P, kv):  # noqa: F811
    """20,000 sequences of which eight have queries, first and last ones among them."""
    import torch

    rng = np.random.default_rng(31)
    B, page, D = 20000, 16, 64
    with_q = {0: 3, 1: 40, 511: 1, 640: 2, 9999: 130, 10000: 1, 19998: 5, 19999: 60}
    lens = {b: n + int(rng.integers(0, 200)) for b, n in with_q.items()}
    s = Paged(P, rng, list(lens.values()), 2, D, page, kv)
    table = np.full((B, s.table.shape[1]), -1, np.int32)
    for i, b in enumerate(with_q):
        table[b] = s.table[i]
    all_lens = rng.integers(0, 300, B)
    nq = np.zeros(B, np.int64)
    for b, n in with_q.items():
        nq[b], all_lens[b] = n, lens[b]
    cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    q = _values(rng, (cu[-1], 8, D), "bf16")
    lse = torch.empty(cu[-1], 8, device="cuda")
    out = P.attn_chunk(_dev(q, "bf16"), s.cache, _pages(table), _i32(all_lens), torch.from_numpy(cu).cuda(), lse=lse)
    P.device_check()
    _check(s, q, list(with_q.values()), _host(out), _host(lse))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_code_and_any_scale(P, D):  # noqa: F811
    """Codes of -128, scales that are 0, negative, tiny and large: a row stands for code times scale."""
    import torch

    rng = np.random.default_rng(D + 1)
    n, nq, Hq, page = 300, 40, 3, 16
    pages = -(-n // page)
    cache = P.KVCache.empty(pages, 1, page, D, torch.int8)
    codes = rng.integers(-128, 128, (2, pages, 1, page, D)).astype(np.int8)
    codes[:, 0, 0, 0] = np.resize(np.arange(-128, 128), (2, D))
    scales = rng.choice([0.01, 0.02, -0.01, 0.0, 1e-30, 0.5], (2, pages, 1, page)).astype(np.float32)
    scales[1, 3] = 1e30
    for t, x in ((cache.k, codes[0]), (cache.v, codes[1]), (cache.k_scale, scales[0]), (cache.v_scale, scales[1])):
        t.copy_(torch.from_numpy(x).cuda())
    k, v = ((codes[i].astype(np.float64) * scales[i][..., None])[:, 0].reshape(-1, D)[:n] for i in range(2))
    q = R.bf16(_values(rng, (nq, Hq, D), "bf16") / 4)
    lse = torch.empty(nq, Hq, device="cuda")
    for window, sinks in ((0, 0), (60, 4)):
        out = _host(P.attn_chunk(_dev(q, "bf16"), cache, _pages(np.arange(pages, dtype=np.int32)[None]), _i32([n]),
                                 _i32((0, nq)), window=window, sinks=sinks, lse=lse))
        for h in range(Hq):
            seen = _sees(n - nq + np.arange(nq), np.arange(n), window, sinks)
            ref = R.attend(q[:, h], k, v, D ** -0.5, seen)
            R.check(out[:, h], _host(lse)[:, h], ref, True, True, f"head {h}")


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_outputs_and_workspaces_at_16_bytes(P, kv):  # noqa: F811
    import torch

    rng = np.random.default_rng(33)
    s = Paged(P, rng, [3000], 2, 128, 16, kv)
    q = _dev(_values(rng, (30, 6, 128), "bf16"), "bf16")
    cu = _i32((0, 30))
    want = P.attn_chunk(q, s.cache, s.table_d, s.lens_d, cu)
    need = P.attn_chunk_workspace_bytes(1, 30, 6, 2, 128, P.PTQ_BF16)
    room = torch.empty(30 * 6 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((need + 64,), 99, dtype=torch.uint8, device="cuda")
    out = room[8:].view(30, 6, 128)
    P.attn_chunk(q, s.cache, s.table_d, s.lens_d, cu, out=out, workspace=ws[16:16 + need])
    assert torch.equal(out, want)
    assert (ws[:16] == 99).all() and (ws[16 + need:] == 99).all()


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_graphs_of_two_streams_with_default_buffers(P, kv):  # noqa: F811
    """Captured calls that allocate their own workspaces, replayed on two streams at once."""
    import torch

    rng = np.random.default_rng(34)
    s = Paged(P, rng, [4000, 500], 2, 128, 64, kv)
    cu = _i32((0, 4, 70))
    qs = [_dev(_values(rng, (70, 8, 128), "bf16"), "bf16") for _ in range(2)]
    want = [P.attn_chunk(q, s.cache, s.table_d, s.lens_d, cu) for q in qs]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in qs]
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(P.attn_chunk(q, s.cache, s.table_d, s.lens_d, cu))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    P.device_check()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_the_last_tile_of_a_page_is_another_sequences(P):  # noqa: F811
    """Tokens past a sequence's end, in its last page, hold another's values or none at all."""
    rng = np.random.default_rng(35)
    for kv in ("bf16", "i8"):
        for D in (64, 128, 256):
            s = Paged(P, rng, [1100, 65, 1], 1, D, 256, kv)      # (what no token has written is NaN)
            nq = (200, 5, 1)
            q = _values(rng, (206, 3, D), "bf16")
            out, lse = _run(P, s, q, nq)
            _check(s, q, nq, out, lse, rows=12, rng=rng)


@pytest.mark.parametrize("kv,act", [("bf16", "bf16"), ("i8", "bf16"), ("i8", "f32"), ("bf16", "f32")])
def test_appending_and_attention_in_a_row(P, kv, act):  # noqa: F811
    """A prompt in chunks and then token by token, norms and rotation on the way, captured and
    replayed: each step's outputs against 64-bit arithmetic over what the cache holds by definition."""
    import torch

    rng = np.random.default_rng(36)
    Hq, Hkv, D, page, window, sinks = 6, 2, 64, 16, 50, 3
    total, chunks = 90, (37, 1, 30)
    x = _values(rng, (total, Hq + 2 * Hkv, D), act)
    inv = (1e4 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
    gq, gk = (1 + 0.1 * rng.standard_normal((2, D))).astype(np.float32)
    pos = np.arange(total, dtype=np.int32)[None]
    q64, qsize = rope_ref.turned(x[:, :Hq], gq, 1e-6, pos, inv, None, False)
    k64, ksize = rope_ref.turned(x[:, Hq:Hq + Hkv], gk, 1e-6, pos, inv, None, False)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    rope = P.Rope(up(inv), q_gain=up(gq), k_gain=up(gk))
    cache = P.KVCache.empty(8, Hkv, page, D, _torch(kv))
    table = up(rng.permutation(8)[None].astype(np.int32))
    xd = _dev(x, act)
    t = torch.arange(total, device="cuda")
    slots = (table[0][t // page] * page + t % page).to(torch.int32)

    def step(at, n, single):
        q, k, v = xd[at:at + n].split((Hq, Hkv, Hkv), 1)
        qt = P.kv_append(cache, rope, k, v, slots[at:at + n], t[at:at + n].to(torch.int32), q=q)
        lens = _i32([at + n])
        if single:
            return qt, P.attn_decode(qt, cache, table, lens, window=window, sinks=sinks)
        return qt, P.attn_chunk(qt.bfloat16(), cache, table, lens, _i32((0, n)), window=window, sinks=sinks)

    at = 0
    for n in chunks + (1,) * (total - sum(chunks)):
        single = n == 1
        qt, out = step(at, n, single)
        qt, out = _host(qt if single else qt.bfloat16()), _host(out)
        # the queries are the definition's, the keys and values are what the cache stands for
        # (an fp32 chunk's queries are rounded to bf16 for attn_chunk: one rounding either way)
        limit = rope_ref.bound(q64[at:at + n], qsize[at:at + n], act == "bf16" or not single)
        assert (np.abs(qt - q64[at:at + n]) <= limit).all()
        ck, cv = (_host(a) for a in P.kv_read(cache, slots[:at + n], dtype=torch.float32))
        for h in range(Hkv):
            limit = rope_ref.code_bound(k64[:at + n, h], ksize[:at + n, h]) if kv == "i8" else rope_ref.bound(
                k64[:at + n, h], ksize[:at + n, h], True)
            assert (np.abs(ck[:, h] - k64[:at + n, h]) <= limit).all()
        seen = _sees(at + np.arange(n), np.arange(at + n), window, sinks)
        for h in range(Hq):
            ref = R.attend(qt[:, h], ck[:, h * Hkv // Hq], cv[:, h * Hkv // Hq], D ** -0.5, seen)
            R.check(out[:, h], None, ref, act == "bf16" or not single, not single, f"token {at} head {h}")
        at += n
