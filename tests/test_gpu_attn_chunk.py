"""Attention of chunks over the paged cache (attn_chunk), and windows of chunks
and of single tokens (attn_decode), on the GPU, against plain 64-bit
arithmetic (tests/attn_ref.py)."""
import numpy as np
import pytest

import attn_ref as R
from test_gpu_attn_decode import Paged, _dev, _host, _stored, _torch, _values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import ternary_weight_ptq1_gb300 as P

    P.load()
    return P


def _sees(p, j, window, sinks):
    """Which tokens j the queries at positions p see."""
    p, j = np.asarray(p)[:, None], np.asarray(j)[None]
    s = j <= p
    if window:
        s &= (j > p - window) | (j < sinks)
    return s


def _i32(x):
    import torch

    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _pages(table):
    import torch

    return torch.from_numpy(table).cuda()


def _run(P, s, q, nq, first=0, after=0, **kw):
    """attn_chunk for nq[b] queries of each sequence, `first` rows before them and
    `after` behind in q, which belong to no sequence."""
    import torch

    cu = first + np.concatenate([[0], np.cumsum(nq)])
    assert cu[-1] + after == len(q)
    qd = q if isinstance(q, torch.Tensor) else _dev(q, "bf16")
    out = torch.full(tuple(qd.shape), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(tuple(qd.shape[:2]), 7.0, device="cuda")
    P.attn_chunk(qd, s.cache, s.table_d, s.lens_d, _i32(cu), out=out, lse=lse, **kw)
    P.device_check()
    return _host(out), _host(lse)


def _check(s, q, nq, out, lse, window=0, sinks=0, first=0, scale=None, rows=None, rng=None, p_bf16=True):
    """Every row, or `rows` random ones of each sequence, against the definition."""
    Hkv, D = s.cache.kv_heads, s.cache.head_dim
    G, scale, at = q.shape[1] // Hkv, D ** -0.5 if scale is None else scale, first
    for b, n in enumerate(nq):
        k, v = _stored(s.k[b], s.kv), _stored(s.v[b], s.kv)
        use = np.arange(n) if rows is None or n <= rows else np.sort(rng.permutation(n)[:rows])
        if rows is not None and n > rows:
            use[0], use[-1] = 0, n - 1
        seen = _sees(s.lens[b] - n + use, np.arange(s.lens[b]), window, sinks)
        for h in range(Hkv):
            for g in range(G):
                hq = h * G + g
                ref = R.attend(q[at + use, hq], k[:, h], v[:, h], scale, seen)
                R.check(out[at + use, hq], lse[at + use, hq], ref, True, p_bf16, f"seq {b} head {hq}")
        at += n


# (sequences' cached tokens, their new ones, query heads, kv heads, head_dim, page, window, sinks)
CASES = [
    ((1,), (1,), 1, 1, 64, 16, 0, 0), ((5,), (5,), 5, 1, 128, 16, 0, 0), ((130,), (4,), 5, 1, 128, 24, 0, 0),
    ((300, 1, 77), (7, 1, 77), 8, 2, 128, 64, 0, 0), ((129, 128, 127), (1, 2, 3), 16, 1, 64, 100, 0, 0),
    ((700,), (300,), 10, 2, 128, 16, 0, 0), ((513, 90), (200, 90), 7, 1, 64, 8, 0, 0),
    ((400, 33), (130, 33), 6, 1, 256, 16, 0, 0), ((260,), (2,), 12, 2, 256, 64, 0, 0), ((50, 60), (20, 31), 20, 1, 64, 7, 0, 0),
    ((40,), (40,), 3, 3, 128, 1, 0, 0), ((1000,), (9,), 4, 1, 128, 256, 0, 0),
    # windows and first tokens
    ((300,), (1,), 5, 1, 128, 16, 1, 0), ((300,), (40,), 5, 1, 128, 16, 1, 1), ((700, 20), (200, 20), 5, 1, 128, 16, 64, 4),
    ((600,), (5,), 8, 1, 128, 64, 128, 130), ((900,), (300,), 4, 2, 64, 24, 200, 3), ((520, 70), (70, 70), 6, 1, 256, 64, 100, 5),
    ((300,), (300,), 2, 1, 128, 16, 40, 300), ((300,), (300,), 2, 1, 128, 16, 299, 2), ((200,), (60,), 4, 1, 64, 16, 2 ** 31 - 1, 2 ** 31 - 1),
    ((1500,), (700,), 1, 1, 128, 16, 33, 64),
    # fewer cached tokens than queries: the first ones see none
    ((3, 0, 20), (10, 4, 21), 5, 1, 128, 16, 0, 0), ((140, 0), (300, 0), 5, 1, 128, 16, 50, 4), ((60,), (200,), 6, 1, 256, 16, 0, 0),
    ((0, 0), (3, 200), 4, 2, 64, 16, 0, 0),
]


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_against_the_definition(P, case, kv):
    lens, nq, Hq, Hkv, D, page, window, sinks = case
    rng = np.random.default_rng(len(str(case)))
    s = Paged(P, rng, list(lens), Hkv, D, page, kv, act="bf16")
    q = _values(rng, (sum(nq), Hq, D), "bf16")
    out, lse = _run(P, s, q, nq, window=window, sinks=sinks)
    _check(s, q, nq, out, lse, window, sinks, rows=24, rng=rng)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_sequences_and_many(P, D, kv):
    """Work that is cut between CTAs in the middle of sequences, beside short ones."""
    rng = np.random.default_rng(D)
    lens, nq = [9000, 40, 0, 3000, 1], [5, 40, 0, 600, 1]
    s = Paged(P, rng, lens, 2, D, 64, kv, act="bf16")
    q = _values(rng, (sum(nq), 10, D), "bf16")
    for window, sinks in ((0, 0), (1000, 4)):
        out, lse = _run(P, s, q, nq, window=window, sinks=sinks)
        _check(s, q, nq, out, lse, window, sinks, rows=3, rng=rng)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_many_sequences_of_few_tokens(P, kv):
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 500, 700)]
    nq = [int(rng.integers(0, min(5, n) + 1)) for n in lens]
    s = Paged(P, rng, lens, 2, 64, 16, kv, act="bf16")
    q = _values(rng, (sum(nq), 4, 64), "bf16")
    out, lse = _run(P, s, q, nq, window=100, sinks=2)
    _check(s, q, nq, out, lse, 100, 2)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 40, 8), (256, 24, 4), (64, 28, 4)])
def test_many_runs_of_every_kind(P, D, Hq, Hkv, kv):
    """Many runs a CTA, of one Q tile and two, with one tile of keys and several, in any order."""
    rng = np.random.default_rng(23)
    lens, nq = [], []
    for _ in range(60):
        n = int(rng.choice([1, 2, 20, 30, 55, 77, 130, 260, 300]))
        nq.append(n)
        lens.append(max(0, n + int(rng.choice([0, 0, -1, 1, 100, 127, 300, -n // 2]))))
    s = Paged(P, rng, lens, Hkv, D, 16, kv)
    q = _values(rng, (sum(nq), Hq, D), "bf16")
    for window, sinks in ((0, 0), (90, 2)):
        first = None
        for _ in range(3):
            out, lse = _run(P, s, q, nq, window=window, sinks=sinks)
            assert first is None or ((out == first[0]).all() and (lse == first[1]).all())
            first = out, lse
        at = np.concatenate([[0], np.cumsum(nq)])
        for b in rng.permutation(60)[:12]:
            k, v = _stored(s.k[b], kv), _stored(s.v[b], kv)
            hq = int(rng.integers(Hq))
            i = rng.integers(nq[b], size=3)
            seen = _sees(lens[b] - nq[b] + i, np.arange(lens[b]), window, sinks)
            ref = R.attend(q[at[b] + i, hq], k[:, hq * Hkv // Hq], v[:, hq * Hkv // Hq], D ** -0.5, seen)
            R.check(out[at[b] + i, hq], lse[at[b] + i, hq], ref, True, True, f"seq {b} head {hq}")


def test_rows_of_no_sequence_are_left(P):
    rng = np.random.default_rng(6)
    s = Paged(P, rng, [100, 30], 1, 128, 16, "bf16")
    nq = (9, 30)
    q = _values(rng, (39 + 5 + 70, 5, 128), "bf16")
    out, lse = _run(P, s, q, nq, first=5, after=70)
    _check(s, q, nq, out, lse, first=5)
    for rows in (slice(0, 5), slice(44, None)):
        assert (out[rows] == 5.0).all() and (lse[rows] == 7.0).all()


def test_offsets_count_into_the_queries(P):
    import torch

    rng = np.random.default_rng(7)
    s = Paged(P, rng, [64, 64], 1, 64, 16, "bf16")
    q = _dev(_values(rng, (20, 4, 64), "bf16"), "bf16")
    good = P.attn_chunk(q, s.cache, s.table_d, s.lens_d, _i32((0, 8, 20)))
    wild = P.attn_chunk(q, s.cache, s.table_d, s.lens_d, _i32((-5, 8, 1000)))
    assert torch.equal(good, wild)
    long = torch.tensor([10 ** 9, 64], dtype=torch.int32, device="cuda")       # counts as the table's
    assert torch.equal(good, P.attn_chunk(q, s.cache, s.table_d, long, _i32((0, 8, 20))))


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
def test_hidden_keys_and_values_have_no_effect(P, kv, window, sinks, what):
    """Tokens that are not finite, hidden from some rows of a tile and seen by others."""
    rng = np.random.default_rng(8)
    lens, nq = [333, 90], (150, 7)
    for D, Hq in ((128, 5), (256, 6), (64, 7)):
        s = Paged(P, rng, lens, 1, D, 16, kv, act="bf16")
        q = _values(rng, (sum(nq), Hq, D), "bf16")
        clean = _run(P, s, q, nq, window=window, sinks=sinks)
        ends = np.cumsum(lens)
        at = [150, 200, 250, 332, lens[0] + 20, lens[0] + 86]   # tokens, counted over both sequences
        for store, codes, scale in ((0, s.cache.k, s.cache.k_scale), (1, s.cache.v, s.cache.v_scale)):
            keep = codes.clone(), None if scale is None else scale.clone()
            for t in at:
                slot = int(s.slots[t])
                if kv == "i8":
                    scale[slot // 16, :, slot % 16] = what
                else:
                    codes[slot // 16, :, slot % 16, 3] = what
            out, lse = _run(P, s, q, nq, window=window, sinks=sinks)
            for b in range(2):
                p = lens[b] - nq[b] + np.arange(nq[b])
                mine = [t - (ends[b - 1] if b else 0) for t in at if (t >= lens[0]) == (b == 1)]
                hit = _sees(p, mine, window, sinks).any(1)
                rows = slice(0, nq[0]) if b == 0 else slice(nq[0], None)
                o, l = out[rows], lse[rows]
                assert (o[~hit] == clean[0][rows][~hit]).all() or np.abs(o[~hit] - clean[0][rows][~hit]).max() <= 2.0 ** -6
                assert np.isfinite(o[~hit]).all() and np.allclose(l[~hit], clean[1][rows][~hit], 0, 1e-4)
                if store == 1:      # a seen value spoils its dimension (int8: its row), and the scores not at all
                    spoilt = ~np.isfinite(o[hit])
                    assert spoilt[..., 3].all() and (kv == "i8" or not np.delete(spoilt, 3, -1).any())
                    assert np.allclose(l[hit], clean[1][rows][hit], 0, 1e-4)
                elif np.isnan(what):
                    assert np.isnan(o[hit]).all() and np.isnan(l[hit]).all()
            codes.copy_(keep[0])
            if scale is not None:
                scale.copy_(keep[1])


def test_infinite_keys_count_as_the_formula_says(P):
    """A key whose score is -infinity weighs nothing; a row of such scores alone sees none."""
    rng = np.random.default_rng(9)
    s = Paged(P, rng, [40], 1, 64, 16, "bf16")
    q = R.bf16(np.abs(_values(rng, (3, 2, 64), "bf16")) + np.float32(0.5))     # as the call takes it
    slot = int(s.slots[11])
    s.cache.k[slot // 16, :, slot % 16, 0] = -np.inf
    out, lse = _run(P, s, q, (3,))
    for h in range(2):
        seen = _sees(37 + np.arange(3), np.arange(40), 0, 0)
        seen[:, 11] = False
        ref = R.attend(q[:, h], s.k[0][:, 0], s.v[0][:, 0], 0.125, seen)
        R.check(out[:, h], lse[:, h], ref, True, True)
    s.cache.k[..., 0] = -np.inf
    out, lse = _run(P, s, q, (3,))
    assert (out == 0).all() and np.isneginf(lse).all()


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_pages_outside_the_cache(P, kv, D):
    """A bad entry makes the rows NaN that see one of its tokens; others it does not touch."""
    rng = np.random.default_rng(10)
    lens, nq = [330, 100], (200, 100)
    s = Paged(P, rng, lens, 2, D, 16, kv, act="bf16")
    q = _values(rng, (300, 4, D), "bf16")
    for window, sinks in ((0, 0), (40, 0)):
        clean = _run(P, s, q, nq, window=window, sinks=sinks)
        for bad in (-1, 10 ** 6, 2 ** 31 - 1):
            t = s.table.copy()
            t[0, 17], t[0, 9] = bad, bad                   # tokens 272 .. 287 and 144 .. 159
            s.table_d.copy_(_pages(t))
            out, lse = _run(P, s, q, nq, window=window, sinks=sinks)
            p = 130 + np.arange(200)
            hit = np.concatenate([_sees(p, list(range(144, 160)) + list(range(272, 288)), window, sinks).any(1),
                                  np.zeros(100, bool)])
            assert np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
            assert np.abs(out[~hit] - clean[0][~hit]).max() <= 2.0 ** -6 and np.allclose(lse[~hit], clean[1][~hit], 0, 1e-4)
        s.table_d.copy_(_pages(s.table))
    # entries that no query sees may be anything
    t = s.table.copy()
    t[0, :18] = -1
    s.table_d.copy_(_pages(t))
    out, lse = _run(P, s, q[:5], (2, 3), window=40, sinks=0)
    assert np.isfinite(out).all()


def test_large_values_do_not_overflow(P):
    """Outputs near the largest bf16 value: weights larger than one may not spoil the sums."""
    rng = np.random.default_rng(11)
    for D, Hq in ((128, 5), (256, 6), (64, 7)):
        s = Paged(P, rng, [500], 1, D, 16, "bf16")
        s.v[0] = R.bf16(np.sign(s.v[0][:1, :, :]) * np.float32(3e38) * np.ones_like(s.v[0]))
        s.k[0] = R.bf16(s.k[0] * np.linspace(0.1, 6, 500)[:, None, None].astype(np.float32))   # maxima that grow
        import torch
        P.kv_write(s.cache, _dev(s.k[0], "bf16"), _dev(s.v[0], "bf16"), torch.from_numpy(s.slots).cuda())
        q = _values(rng, (200, Hq, D), "bf16")
        out, lse = _run(P, s, q, (200,))
        assert np.isfinite(out).all()
        _check(s, q, (200,), out, lse, rows=6, rng=rng)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_strided_queries_scale_and_none_given(P, kv):
    import torch

    rng = np.random.default_rng(12)
    s = Paged(P, rng, [222, 31], 2, 128, 16, kv)
    nq = (60, 4)
    x = _dev(_values(rng, (64, 14, 128), "bf16"), "bf16")
    q = x[:, 2:12]
    assert not q.is_contiguous()
    out, lse = _run(P, s, q, nq, scale=0.21)
    _check(s, _host(q).astype(np.float32), nq, out, lse, scale=0.21)
    alone = P.attn_chunk(q, s.cache, s.table_d, s.lens_d, _i32((0, 60, 64)), scale=0.21)
    assert torch.equal(alone.double().cpu(), torch.from_numpy(out))


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_results_repeat_and_workspaces_may_hold_anything(P, kv, D):
    import torch

    rng = np.random.default_rng(13)
    lens, nq = [5000, 300], (3, 200)
    s = Paged(P, rng, lens, 2, D, 64, kv)
    q = _dev(_values(rng, (203, 8, D), "bf16"), "bf16")
    need = P.attn_chunk_workspace_bytes(2, 203, 8, 2, D, P.PTQ_BF16)
    got = []
    for fill in (0, 255, 127):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        ws[need:] = 170
        got.append(P.attn_chunk(q, s.cache, s.table_d, s.lens_d, _i32((0, 3, 203)), workspace=ws[:need] if need else None))
        assert (ws[need:] == 170).all()
    assert all(torch.equal(g, got[0]) for g in got)


def test_a_graph_follows_lengths_offsets_and_tables(P):
    import torch

    rng = np.random.default_rng(14)
    s = Paged(P, rng, [3000, 200], 2, 128, 16, "i8")
    q = _values(rng, (40, 10, 128), "bf16")
    qd, out, lse = _dev(q, "bf16"), torch.empty(40, 10, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(40, 10, device="cuda")
    cu, lens = _i32((0, 1, 40)), s.lens_d.clone()
    ws = torch.empty(max(1, P.attn_chunk_workspace_bytes(2, 40, 10, 2, 128, P.PTQ_BF16)), dtype=torch.uint8, device="cuda")
    call = lambda: P.attn_chunk(qd, s.cache, s.table_d, lens, cu, window=500, sinks=2, out=out, lse=lse, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    full_k, full_v, full = s.k, s.v, s.lens
    for new, nq in (((3000, 200), (1, 39)), ((700, 90), (30, 10)), ((12, 200), (5, 35))):
        lens.copy_(_i32(new))
        cu.copy_(_i32((0, nq[0], 40)))
        g.replay()
        torch.cuda.synchronize()
        s.lens, s.k, s.v = list(new), [k[:n] for k, n in zip(full_k, new)], [v[:n] for v, n in zip(full_v, new)]
        _check(s, q, nq, _host(out), _host(lse), 500, 2, rows=5, rng=rng)
    s.k, s.v, s.lens = full_k, full_v, full
    P.device_check()


def test_two_streams_at_once(P):
    import torch

    rng = np.random.default_rng(15)
    s = Paged(P, rng, [2000, 900], 2, 128, 64, "bf16")
    qs = [_dev(_values(rng, (64, 8, 128), "bf16"), "bf16") for _ in range(2)]
    cu = _i32((0, 10, 64))
    want = [P.attn_chunk(q, s.cache, s.table_d, s.lens_d, cu) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[P.attn_chunk(q, s.cache, s.table_d, s.lens_d, cu, stream=st) for q, st in zip(qs, streams)] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, want):
            assert torch.equal(g, w)


def test_rows_past_32_bits_of_offset(P):
    """Pages whose offsets pass 2^32 bytes and 2^31 values."""
    import torch

    for kv, pages in (("bf16", 2 ** 19 + 5), ("i8", 2 ** 19 + 5)):
        rng = np.random.default_rng(16)
        page, D = 64, 128
        cache = P.KVCache.empty(pages, 1, page, D, _torch(kv))       # 2^32 values and more
        table = np.array([[pages - 1, 3, pages - 2, 2 ** 18, pages - 3]], np.int32)
        n, nq = 300, 20
        k, v = (_values(rng, (n, 1, D), "bf16") for _ in range(2))
        j = np.arange(n)
        slots = (table[0, j // page].astype(np.int64) * page + j % page).astype(np.int32)
        P.kv_write(cache, _dev(k, "bf16"), _dev(v, "bf16"), torch.from_numpy(slots).cuda())
        s = type("S", (), {})()
        s.cache, s.table_d, s.lens_d, s.lens, s.k, s.v, s.kv = cache, _pages(table), _i32([n]), [n], [k], [v], kv
        q = _values(rng, (nq, 5, D), "bf16")
        out, lse = _run(P, s, q, (nq,))
        _check(s, q, (nq,), out, lse)
        del cache, s
        torch.cuda.empty_cache()


def test_chunk_of_one_token_is_decode(P):
    rng = np.random.default_rng(17)
    lens = [1, 40, 700, 0, 2500]
    for kv in ("bf16", "i8"):
        s = Paged(P, rng, lens, 2, 128, 16, kv)
        q = _values(rng, (5, 10, 128), "bf16")
        for window, sinks in ((0, 0), (300, 4)):
            out, lse = _run(P, s, q, [1] * 5, window=window, sinks=sinks)
            import torch
            l2 = torch.empty(5, 10, device="cuda")
            o2 = _host(P.attn_decode(_dev(q, "bf16"), s.cache, s.table_d, s.lens_d, lse=l2, window=window, sinks=sinks))
            assert np.abs(out - o2).max() <= 2.0 ** -6 and np.allclose(lse, _host(l2), 0, 1e-4)


# ---- one new token under a window ------------------------------------------------------

WINDOWS = [((300, 1, 5, 0, 64, 65), 5, 1, 128, 16, 64, 0), ((3000, 70, 900), 8, 2, 128, 64, 1000, 4), ((700,), 5, 1, 128, 16, 1, 0),
           ((700, 40), 4, 4, 64, 24, 100, 33), ((900, 2), 6, 1, 256, 64, 130, 7), ((500,), 16, 1, 128, 100, 77, 1),
           ((129, 130, 131, 132, 133), 2, 1, 64, 8, 128, 3), ((400,), 3, 1, 128, 7, 399, 5), ((400,), 3, 1, 128, 16, 400, 5),
           ((9000, 8000), 20, 2, 128, 64, 5000, 50), ((300,), 5, 1, 128, 16, 10, 2 ** 31 - 1), ((600, 600), 12, 1, 64, 256, 200, 600),
           ((20000,), 5, 1, 128, 16, 300, 40)]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("case", WINDOWS, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_window_of_one_token(P, case, act, kv):
    import torch

    lens, Hq, Hkv, D, page, window, sinks = case
    rng = np.random.default_rng(len(str(case)))
    s = Paged(P, rng, list(lens), Hkv, D, page, kv, act=act)
    q = _values(rng, (len(lens), Hq, D), act)
    lse = torch.full((len(lens), Hq), 7.0, device="cuda")
    out = _host(P.attn_decode(_dev(q, act), s.cache, s.table_d, s.lens_d, lse=lse, window=window, sinks=sinks))
    _check(s, q, [1] * len(lens), out, _host(lse), window, sinks, p_bf16=False) if act == "bf16" else None
    if act == "f32":
        G = Hq // Hkv
        for b, n in enumerate(lens):
            k, v = _stored(s.k[b], kv), _stored(s.v[b], kv)
            seen = _sees([n - 1], np.arange(n), window, sinks)
            for h in range(Hq):
                ref = R.attend(q[b, h][None], k[:, h // G], v[:, h // G], D ** -0.5, seen)
                R.check(out[b, h][None], _host(lse)[b, h][None], ref, False, False, f"seq {b} head {h}")


def test_a_window_hides_tokens_and_pages(P):
    """Hidden tokens that are not finite and hidden entries that are no pages have no effect."""
    rng = np.random.default_rng(18)
    for kv in ("bf16", "i8"):
        s = Paged(P, rng, [1000], 1, 128, 16, kv, act="f32")
        q = _values(rng, (1, 5, 128), "f32")
        run = lambda: _host(P.attn_decode(_dev(q), s.cache, s.table_d, s.lens_d, window=100, sinks=3))  # noqa: E731
        clean = run()
        for t in list(range(3, 900)):
            slot = int(s.slots[t])
            (s.cache.k if kv == "bf16" else s.cache.k_scale)[slot // 16, :, slot % 16] = np.nan
            (s.cache.v if kv == "bf16" else s.cache.v_scale)[slot // 16, :, slot % 16] = np.inf
        t = s.table.copy()
        t[0, 1:56] = -9                     # tokens 16 .. 895
        s.table_d.copy_(_pages(t))
        assert (run() == clean).all()
        t[0, 0] = 10 ** 8
        s.table_d.copy_(_pages(t))
        assert np.isnan(run()).all()
