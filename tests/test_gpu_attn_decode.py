"""The paged key-value cache and the attention of one new token over it, on
the GPU, against plain 64-bit arithmetic (tests/attn_ref.py)."""
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


def _torch(kind):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8}[kind]


def _dev(x, kind="f32"):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(_torch(kind))


def _host(t):
    return t.double().cpu().numpy()


def _values(rng, shape, act):
    x = rng.standard_normal(shape).astype(np.float32)
    return R.bf16(x) if act == "bf16" else x


def _stored(x, kv):
    """What a cache of type kv holds for the fp32 rows x."""
    if kv == "bf16":
        return R.bf16(x)
    c, s = R.quantise(x)
    return c.astype(np.float64) * s[..., None].astype(np.float64)


class Paged:
    """Sequences of random keys and values in a cache of shuffled pages, with
    NaN (bf16) or extreme codes and NaN scales (int8) wherever no token is."""

    def __init__(self, P, rng, lens, Hkv, D, page, kv, act="bf16", spare=3, width=None):
        import torch

        used = [-(-n // page) for n in lens]
        pages = max(1, sum(used) + spare)
        self.cache = P.KVCache.empty(pages, Hkv, page, D, _torch(kv))
        if kv == "bf16":
            self.cache.k.fill_(float("nan"))
            self.cache.v.fill_(float("nan"))
        else:
            self.cache.k.fill_(-128)
            self.cache.v.fill_(-128)
            self.cache.k_scale.fill_(float("nan"))
            self.cache.v_scale.fill_(float("nan"))
        order = rng.permutation(pages)
        width = max(1, max(used)) if width is None else width
        table = np.full((len(lens), width), -7, np.int32)
        at, slots = 0, []
        for b, n in enumerate(lens):
            table[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
            j = np.arange(n)
            slots.append(table[b, j // page].astype(np.int64) * page + j % page)
        self.lens, self.table = lens, table
        self.k, self.v = ([_values(rng, (n, Hkv, D), act) for n in lens] for _ in range(2))
        self.slots = np.concatenate(slots).astype(np.int32)
        P.kv_write(self.cache, _dev(np.concatenate(self.k), act), _dev(np.concatenate(self.v), act),
                   _dev(self.slots, "f32").to(torch.int32) if len(self.slots) == 0 else
                   torch.from_numpy(self.slots).cuda())
        self.table_d = torch.from_numpy(table).cuda()
        self.lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.kv = kv

    def check(self, q, out, lse, scale, bf16_out, what="", only=None):
        Hkv = self.cache.kv_heads
        G = q.shape[1] // Hkv
        for b in range(len(self.lens)) if only is None else only:
            k, v = _stored(self.k[b], self.kv), _stored(self.v[b], self.kv)
            for h in range(Hkv):
                rows = slice(h * G, h * G + G)
                ref = R.attend(q[b, rows], k[:, h], v[:, h], scale)
                R.check(out[b, rows], lse[b, rows], ref, bf16_out, False, f"{what} seq {b} head {h}")


def _run(P, rng, s, Hq, act, scale=None, **kw):
    import torch

    D = s.cache.head_dim
    q = _values(rng, (len(s.lens), Hq, D), act)
    lse = torch.full((len(s.lens), Hq), 7.0, device="cuda")
    out = P.attn_decode(_dev(q, act), s.cache, s.table_d, s.lens_d, scale=scale, lse=lse, **kw)
    return q, _host(out), _host(lse)


# ---- the cache -------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_write_and_read(P, D, act, kv):
    import torch

    rng = np.random.default_rng(D)
    T, Hkv, page, pages = 37, 3, 5, 11
    x = _values(rng, (T, 2, Hkv, D), act)
    x[3, 0, 1] = 0.0                        # a row of zeros
    x[4, 0, 0] *= 2.0 ** 40
    x[5, 1, 2] *= 2.0 ** -40
    x[6, 0, 0, :] = np.arange(D) - 0.5      # halves, before the scale
    x[6, 0, 0, 0] = 127.0                   # scale 1: exact ties
    x[6, 0, 0, 1:] = np.clip(x[6, 0, 0, 1:], -120, 120)
    if act == "bf16":
        x = R.bf16(x)
    slots = rng.permutation(page * pages)[:T].astype(np.int32)
    slots[7], slots[8] = -1, page * pages   # skipped
    cache = P.KVCache.empty(pages, Hkv, page, D, _torch(kv))
    for t in (cache.k, cache.v):
        t.fill_(77)
    xd = _dev(x, act)                       # k and v are columns of one row: strided
    P.kv_write(cache, xd[:, 0], xd[:, 1], torch.from_numpy(slots).cuda())
    live = np.array([i for i in range(T) if 0 <= slots[i] < page * pages])
    for name, col, codes, scales in (("k", 0, cache.k, cache.k_scale), ("v", 1, cache.v, cache.v_scale)):
        codes = codes.permute(0, 2, 1, 3).reshape(page * pages, Hkv, D)
        if kv == "i8":
            c, s = R.quantise(x[live][:, col])
            scales = scales.permute(0, 2, 1).reshape(page * pages, Hkv)
            np.testing.assert_array_equal(codes.cpu().numpy()[slots[live]], c, err_msg=name)
            np.testing.assert_array_equal(scales.cpu().numpy()[slots[live]], s, err_msg=name)
        else:
            np.testing.assert_array_equal(_host(codes)[slots[live]], R.bf16(x[live][:, col]))
        rest = np.setdiff1d(np.arange(page * pages), slots[live])
        assert (codes[torch.from_numpy(rest).cuda()] == 77).all()
    out = torch.full((T, 2, Hkv, D), 5.0, dtype=_torch(act), device="cuda")
    P.kv_read(cache, torch.from_numpy(slots).cuda(), k=out[:, 0], v=out[:, 1])
    got = _host(out)
    assert np.isnan(got[[7, 8]]).all()
    if kv == "i8":
        c, s = R.quantise(x[live])
        want = c.astype(np.float32) * s[..., None]
    else:
        want = R.bf16(x[live])
    np.testing.assert_array_equal(got[live], R.bf16(want) if act == "bf16" else want)


def test_non_finite_rows_read_back_as_nan(P):
    import torch

    x = np.ones((4, 1, 64), np.float32)
    x[0, 0, 5], x[1, 0, 63], x[2, 0, 0] = np.inf, np.nan, -np.inf
    cache = P.KVCache.empty(1, 1, 4, 64, torch.int8)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    P.kv_write(cache, _dev(x), _dev(x), slots)
    k, v = P.kv_read(cache, slots, dtype=torch.float32)
    for t in (k, v):
        assert torch.isnan(t[:3]).all() and torch.equal(t[3], torch.ones_like(t[3]))


def test_scale_that_underflows(P):
    # the smallest subnormals: 127 levels do not fit under them, the row is zeros
    import torch

    x = np.zeros((2, 1, 64), np.float32)
    x[0, 0, 3], x[1, 0, 9] = 1e-45, 3e-38
    cache = P.KVCache.empty(1, 1, 2, 64, torch.int8)
    P.kv_write(cache, _dev(x), _dev(x), torch.arange(2, dtype=torch.int32, device="cuda"))
    c, s = R.quantise(x)
    np.testing.assert_array_equal(cache.k.cpu().numpy()[0, 0], c[:, 0])
    np.testing.assert_array_equal(cache.k_scale.cpu().numpy()[0, 0], s[:, 0])


def test_nothing_to_write(P):
    import torch

    cache = P.KVCache.empty(1, 2, 4, 64, torch.int8)
    none = torch.empty((0, 2, 64), device="cuda")
    P.kv_write(cache, none, none, torch.empty(0, dtype=torch.int32, device="cuda"))
    k, v = P.kv_read(cache, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert k.shape == v.shape == (0, 2, 64)


# ---- decode attention ------------------------------------------------------------

@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("D,Hkv,G,page", [(64, 2, 1, 16), (128, 2, 5, 64), (256, 1, 6, 24), (128, 1, 8, 7),
                                          (64, 1, 20, 100), (256, 2, 9, 16), (128, 3, 16, 1)])
def test_decode(P, D, Hkv, G, page, act, kv):
    rng = np.random.default_rng([D, G, page])
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 0, 257, 500]
    s = Paged(P, rng, lens, Hkv, D, page, kv, act)
    q, out, lse = _run(P, rng, s, Hkv * G, act)
    s.check(q, out, lse, D ** -0.5, act == "bf16", f"{act} {kv}")


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("n,page", [(1, 16), (777, 16), (5000, 64), (20011, 256)])
def test_one_sequence_split_over_its_length(P, n, page, kv):
    rng = np.random.default_rng(n)
    s = Paged(P, rng, [n], 2, 128, page, kv, "f32")
    q, out, lse = _run(P, rng, s, 10, "f32")
    s.check(q, out, lse, 128 ** -0.5, False, f"{kv} {n}")


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_many_sequences(P, kv):
    # more (sequence, head) pairs than resident CTAs; some long, most short
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 90, 400)]
    lens[17], lens[399] = 3000, 1111
    s = Paged(P, rng, lens, 4, 64, 16, kv, "bf16")
    q, out, lse = _run(P, rng, s, 4, "bf16")
    s.check(q, out, lse, 0.125, True, kv, only=[0, 1, 16, 17, 18, 100, 250, 398, 399] + list(range(200, 230)))


def test_empty_batch_and_empty_tables(P):
    import torch

    cache = P.KVCache.empty(2, 2, 4, 64, torch.bfloat16)
    q = torch.randn(0, 4, 64, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    assert P.attn_decode(q, cache, torch.zeros((0, 3), **i32), torch.zeros(0, **i32)).shape == (0, 4, 64)
    q, lse = torch.randn(3, 4, 64, device="cuda"), torch.zeros(3, 4, device="cuda")
    out = P.attn_decode(q, cache, torch.zeros((3, 0), **i32), torch.full((3,), 9, **i32), lse=lse)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_lengths_outside_the_table(P):
    # below 0 counts as 0, past the table as the table's end
    import torch

    rng = np.random.default_rng(5)
    s = Paged(P, rng, [32, 32, 32], 1, 64, 16, "bf16", "f32")
    s.lens_d = torch.tensor([-5, 2 ** 31 - 1, 33], dtype=torch.int32, device="cuda")
    q, out, lse = _run(P, rng, s, 2, "f32")
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all()
    s.check(q, out, lse, 0.125, False, only=[1, 2])


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_a_page_outside_the_cache_gives_nan_in_its_sequence_alone(P, kv):
    import torch

    rng = np.random.default_rng(6)
    s = Paged(P, rng, [100, 100, 100, 20], 2, 128, 16, kv, "f32")
    s.table_d[1, 3] = s.cache.pages
    s.table_d[2, 6] = -1
    s.table_d[3, 5] = -1                    # not in use
    q, out, lse = _run(P, rng, s, 4, "f32")
    assert np.isnan(out[1:3]).all() and np.isnan(lse[1:3]).all()
    s.check(q, out, lse, 128 ** -0.5, False, only=[0, 3])


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_large_and_small_values(P, act, kv):
    # queries from 2^-30 to 2^12 (scores to the thousands: one key takes all
    # the weight), values whose size differs by 2^60 between tokens
    import torch

    rng = np.random.default_rng(7)
    lens = [70, 129, 300, 45]
    s = Paged(P, rng, lens, 1, 128, 16, kv, act)
    for b, n in enumerate(lens):
        f = 2.0 ** rng.integers(-30, 30, (n, 1, 1))
        s.v[b] = (s.v[b] * f).astype(np.float32)
    P.kv_write(s.cache, _dev(np.concatenate(s.k), act), _dev(np.concatenate(s.v), act),
               torch.from_numpy(s.slots).cuda())
    q = _values(rng, (4, 3, 128), act) * (2.0 ** np.array([-30, 0, 6, 12]))[:, None, None].astype(np.float32)
    lse = torch.empty(4, 3, device="cuda")
    out = P.attn_decode(_dev(q, act), s.cache, s.table_d, s.lens_d, lse=lse)
    s.check(q, _host(out), _host(lse), 128 ** -0.5, act == "bf16", f"{act} {kv}")


def test_zero_values_and_zero_scales(P):
    import torch

    rng = np.random.default_rng(8)
    s = Paged(P, rng, [40, 40], 1, 64, 16, "i8", "f32")
    s.k[0][:], s.v[1][:] = 0, 0
    s.v[0][:17] = 0
    P.kv_write(s.cache, _dev(np.concatenate(s.k)), _dev(np.concatenate(s.v)), torch.from_numpy(s.slots).cuda())
    q, out, lse = _run(P, rng, s, 4, "f32")
    s.check(q, out, lse, 0.125, False)


def test_a_nan_key_makes_its_sequence_nan_alone(P):
    import torch

    rng = np.random.default_rng(9)
    s = Paged(P, rng, [50, 50, 50], 1, 64, 16, "i8", "f32")
    s.k[1][20, 0, 3] = np.nan
    P.kv_write(s.cache, _dev(np.concatenate(s.k)), _dev(np.concatenate(s.v)), torch.from_numpy(s.slots).cuda())
    q, out, lse = _run(P, rng, s, 2, "f32")
    assert np.isnan(out[1]).all() and np.isnan(lse[1]).all()
    s.check(q, out, lse, 0.125, False, only=[0, 2])


def test_strided_queries_scale_stream_and_guards(P):
    import torch

    rng = np.random.default_rng(10)
    s = Paged(P, rng, [200, 3, 90], 2, 128, 16, "i8", "bf16")
    q = _values(rng, (3, 10, 128), "bf16")
    wide = torch.zeros((3, 20, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 4:14] = _dev(q, "bf16")
    buf = torch.full((3 * 10 * 128 + 4096,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = buf[2048:-2048].view(3, 10, 128)
    lse = torch.empty(3, 10, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    need = P.attn_decode_workspace_bytes(3, 10, 2, 128, P.PTQ_BF16)
    ws = torch.full((need + 32,), 0xff, dtype=torch.uint8, device="cuda")   # any contents
    side.wait_stream(torch.cuda.current_stream())
    P.attn_decode(wide[:, 4:14], s.cache, s.table_d, s.lens_d, scale=0.3, out=out, lse=lse, workspace=ws[:need],
                  stream=side)
    side.synchronize()
    s.check(q, _host(out), _host(lse), float(np.float32(0.3)), True)
    assert (buf[:2048] == 9).all() and (buf[-2048:] == 9).all() and (ws[need:] == 0xff).all()


def test_reproducible_and_capturable(P):
    import torch

    rng = np.random.default_rng(11)
    s = Paged(P, rng, [4000, 1, 0, 900, 2500], 4, 128, 64, "i8", "f32")
    q = _dev(_values(rng, (5, 20, 128), "f32"))
    need = P.attn_decode_workspace_bytes(5, 20, 4, 128, P.PTQ_F32)
    ws = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(5, 20, device="cuda")

    def call():
        P.attn_decode(q, s.cache, s.table_d, s.lens_d, out=out, lse=lse, workspace=ws)

    call()
    first, l1 = out.clone(), lse.clone()
    ws.fill_(0x55)
    call()
    assert torch.equal(out, first) and torch.equal(lse, l1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call()
    s.lens_d.copy_(torch.tensor([1, 300, 4000, 0, 64], dtype=torch.int32))    # lengths move between replays
    s.table_d[[0, 1, 2]] = s.table_d[[1, 3, 0]].clone()
    g.replay()
    again, l2 = out.clone(), lse.clone()
    call()
    assert torch.equal(out, again) and torch.equal(lse, l2) and not torch.equal(out, first)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_offsets_past_32_bits(P, kv):
    # pages beyond 2^31 elements (and, in bf16, 2^32 bytes) of one array
    import torch

    D, Hkv, page = 256, 4, 256
    pages = (2 ** 31) // (D * Hkv * page) + 40
    rng = np.random.default_rng(12)
    cache = P.KVCache.empty(pages, Hkv, page, D, _torch(kv))
    n = 600
    table = np.array([[pages - 1, 0, pages - 17]], np.int32)
    j = np.arange(n)
    slots = (table[0, j // page] * page + j % page).astype(np.int32)
    k, v = (_values(rng, (n, Hkv, D), "bf16") for _ in range(2))
    P.kv_write(cache, _dev(k, "bf16"), _dev(v, "bf16"), torch.from_numpy(slots).cuda())
    q = _values(rng, (1, Hkv, D), "bf16")
    lse = torch.empty(1, Hkv, device="cuda")
    out = P.attn_decode(_dev(q, "bf16"), cache, torch.from_numpy(table).cuda(),
                        torch.tensor([n], dtype=torch.int32, device="cuda"), lse=lse)
    back, _ = P.kv_read(cache, torch.from_numpy(slots).cuda(), dtype=torch.float32)
    np.testing.assert_allclose(_host(back), _stored(k, kv), rtol=2e-7, atol=0)
    for h in range(Hkv):
        ref = R.attend(q[0, h:h + 1], _stored(k, kv)[:, h], _stored(v, kv)[:, h], 1 / 16)
        R.check(_host(out)[0, h:h + 1], _host(lse)[0, h:h + 1], ref, True, False)


def test_infinite_keys(P):
    """A key whose score is -infinity counts for nothing, and a row of such keys
    alone is empty; +infinity and infinite values leave no finite row."""
    import torch

    rng = np.random.default_rng(31)
    D, n = 64, 40
    s = Paged(P, rng, [n, n, n, n], 1, D, 16, "bf16", "bf16")
    s.k[0][17, 0, 3] = s.k[1][:, 0, 3] = -np.inf
    s.k[2][17, 0, 3] = np.inf
    s.v[3][17, 0, 5] = np.inf
    P.kv_write(s.cache, _dev(np.concatenate(s.k), "bf16"), _dev(np.concatenate(s.v), "bf16"),
               torch.from_numpy(s.slots).cuda())
    q = R.bf16(rng.standard_normal((4, 2, D)))
    q[:, :, 3] = 1.0
    lse = torch.empty((4, 2), device="cuda")
    out = _host(P.attn_decode(_dev(q, "bf16"), s.cache, s.table_d, s.lens_d, lse=lse))
    lse = _host(lse)
    use = np.arange(n) != 17
    for h in range(2):
        ref = R.attend(q[0, h:h + 1], s.k[0][use, 0], s.v[0][use, 0], D ** -0.5)
        R.check(out[0, h:h + 1], lse[0, h:h + 1], ref, True, False)
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all()
    assert np.isnan(out[2]).all() and np.isnan(lse[2]).all()
    assert (out[3, :, 5] == np.inf).all() and np.isfinite(out[3][:, np.arange(D) != 5]).all()


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("B,Hkv,G,D,width", [(1, 8, 5, 128, 64), (1, 8, 5, 128, 65), (1, 8, 5, 128, 128),
                                             (1, 8, 5, 128, 129), (3, 4, 6, 256, 40), (1, 4, 6, 256, 40),
                                             (40, 1, 3, 64, 40), (86, 1, 3, 64, 40), (2, 2, 20, 64, 40)])
def test_few_sequences_in_clusters_and_in_runs(P, B, Hkv, G, D, width, kv):
    """Both sides of where a cluster of CTAs takes each (sequence, kv head)."""
    rng = np.random.default_rng(41)
    lens = [int(x) for x in rng.integers(0, 600, B)]
    lens[0] = 601
    act = "f32" if G == 5 else "bf16"
    s = Paged(P, rng, lens, Hkv, D, 16, kv, act, width=width)
    q, out, lse = _run(P, rng, s, Hkv * G, act)
    s.check(q, out, lse, D ** -0.5, act == "bf16", only=sorted(set([0, B - 1, B // 2])))
