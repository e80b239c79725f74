"""Head norms with position rotation (qk_rope) and appending to the cache
(kv_append) on the GPU, against 64-bit arithmetic (tests/rope_ref.py)."""
import numpy as np
import pytest

import attn_ref as A
import rope_ref as R

pytestmark = pytest.mark.gpu

EPS = 1e-6


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


def _dev(x, kind=None):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if kind is None else t.to(_torch(kind))


def _host(t):
    return t.double().cpu().numpy()


class Case:
    """Random heads, gains, positions and frequencies of one call."""

    def __init__(self, T, Hq, Hkv, D, rotary, act, axes=1, interleaved=False, norm="qk", far=4096, seed=0):
        r = np.random.default_rng([T, Hq, D, rotary, seed])
        self.T, self.Hq, self.Hkv, self.D, self.act = T, Hq, Hkv, D, act
        x = r.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float32)
        x[0, 0] *= 2.0 ** 20
        x[-1, -1] *= 2.0 ** -20
        self.x = A.bf16(x) if act == "bf16" else x
        half = rotary // 2
        self.inv = (1e4 ** (-np.arange(half) / max(1, half))).astype(np.float32)
        self.pos = r.integers(0, far, (axes, T)).astype(np.int32)
        self.axis = None if axes == 1 else (np.arange(half) % axes).astype(np.int8)
        self.gq, self.gk = ((1 + 0.2 * r.standard_normal(D)).astype(np.float32) if n in norm else None for n in "qk")
        self.interleaved = interleaved

    def rope(self, P):
        up = lambda a: None if a is None else _dev(a)  # noqa: E731
        return P.Rope(up(self.inv), axis=up(self.axis), interleaved=self.interleaved, q_gain=up(self.gq), k_gain=up(self.gk),
                      eps=EPS)

    def parts(self):
        """q, k, v on the GPU: columns of one row."""
        return _dev(self.x, self.act).split((self.Hq, self.Hkv, self.Hkv), 1)

    def ref(self, which):
        x = self.x[:, :self.Hq] if which == "q" else self.x[:, self.Hq:self.Hq + self.Hkv]
        return R.turned(x, self.gq if which == "q" else self.gk, EPS, self.pos, self.inv, self.axis, self.interleaved)

    def positions(self):
        return _dev(self.pos[0] if len(self.pos) == 1 else self.pos)


def _near(y, ref, size, bf16, what=""):
    err, b = np.abs(_host(y) - ref), R.bound(ref, size, bf16)
    i = np.unravel_index(np.argmax(err - b), err.shape)
    assert (err <= b).all(), f"{what}: {err[i]:.3e} at {i}, bound {b[i]:.3e}"


CASES = [dict(T=1, Hq=5, Hkv=1, D=128, rotary=128), dict(T=7, Hq=40, Hkv=8, D=128, rotary=128, axes=3, far=100000),
         dict(T=5, Hq=6, Hkv=2, D=256, rotary=64, norm=""), dict(T=9, Hq=3, Hkv=3, D=64, rotary=64, interleaved=True),
         dict(T=6, Hq=2, Hkv=1, D=256, rotary=256, interleaved=True, axes=2), dict(T=4, Hq=7, Hkv=1, D=64, rotary=24),
         dict(T=3, Hq=20, Hkv=2, D=128, rotary=8, norm="q"), dict(T=3, Hq=1, Hkv=1, D=128, rotary=0, norm="k"),
         dict(T=1024, Hq=5, Hkv=1, D=128, rotary=128, far=2 ** 31 - 1), dict(T=1027, Hq=2, Hkv=3, D=64, rotary=40, axes=2),
         dict(T=1025, Hq=1, Hkv=1, D=256, rotary=256), dict(T=2, Hq=300, Hkv=11, D=64, rotary=64)]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_qk_rope(P, case, act):
    c = Case(act=act, **case)
    q, k, _ = c.parts()
    qo, ko = P.qk_rope(c.rope(P), q, k, c.positions())
    for which, y in (("q", qo), ("k", ko)):
        _near(y, *c.ref(which), act == "bf16", which)


def test_in_place_and_strided_outputs(P):
    import torch

    c = Case(6, 4, 2, 128, 128, "bf16")
    rope, pos = c.rope(P), c.positions()
    q, k, v = c.parts()
    qo, ko = P.qk_rope(rope, q, k, pos)
    before = v.clone()
    P.qk_rope(rope, q, k, pos, q_out=q, k_out=k)            # in the projection's own rows
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, before)
    wide = torch.full((6, 9, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    q2, k2, _ = c.parts()
    P.qk_rope(rope, q2, k2, pos, q_out=wide[:, 1:5], k_out=wide[:, 6:8])
    assert torch.equal(wide[:, 1:5], qo) and torch.equal(wide[:, 6:8], ko)
    assert (wide[:, [0, 5, 8]] == 7).all()


def test_positions_far_and_negative(P):
    """Angles are right wherever the position is: fp32 products would be off by whole turns."""
    c = Case(8, 2, 1, 128, 128, "f32", norm="")
    c.pos = np.array([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, -(10 ** 9), 123456789]], np.int32)
    c.inv[:4] = (1.0, 3.0, 0.7, 1e-30)
    c.inv[4:8] = (-0.5, 100.25, 2.0 ** -140, 0.0)
    q, k, _ = c.parts()
    qo, ko = P.qk_rope(c.rope(P), q, k, c.positions())
    # fp64 products of 2^31 and 100 are off by 2^-15: more than fp32 allows, so the reference reduces exactly
    from fractions import Fraction

    def arctan_of_one_over(n):                 # to 200 bits
        term, total, k = Fraction(1, n), Fraction(0), 0
        while term > Fraction(1, 1 << 200):
            total += (-1) ** k * term / (2 * k + 1)
            term /= n * n
            k += 1
        return Fraction(int(total * (1 << 200)), 1 << 200)
    two_pi = 8 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239))     # Machin's formula

    def exact(x):
        x = np.array(x, np.float64)
        size, half = np.abs(x), 64
        for i in range(half):
            turns = [float((Fraction(int(p)) * Fraction(float(c.inv[i])) / two_pi) % 1) for p in c.pos[0]]
            t = 2 * np.pi * np.array(turns)
            cs, sn = np.cos(t)[:, None], np.sin(t)[:, None]
            a, b = x[..., i].copy(), x[..., i + half].copy()
            x[..., i], x[..., i + half] = a * cs - b * sn, b * cs + a * sn
            size[..., i] = size[..., i + half] = np.abs(a) + np.abs(b)
        return x, size
    _near(qo, *exact(c.x[:, :2]), False, "q")
    _near(ko, *exact(c.x[:, 2:3]), False, "k")


def test_pairs_of_no_axis_and_frequencies_that_are_not_finite(P):
    import torch

    c = Case(3, 2, 2, 64, 64, "f32", axes=2, norm="")
    c.axis[3], c.axis[5], c.axis[7] = 2, -1, 127
    q, k, _ = c.parts()
    qo, _ = P.qk_rope(c.rope(P), q, k, c.positions())
    _near(qo, *c.ref("q"), False)
    for i in (3, 5, 7):
        assert torch.equal(qo[..., i], q[..., i]) and torch.equal(qo[..., i + 32], q[..., i + 32])
    c.inv[2] = np.inf
    qo, _ = P.qk_rope(c.rope(P), q, k, c.positions())
    y = _host(qo)
    assert np.isnan(y[..., [2, 34]]).all() and np.isfinite(np.delete(y, [2, 34], -1)).all()


def test_rows_of_zeros_large_and_infinite_values(P):
    c = Case(4, 2, 1, 128, 128, "f32")
    c.x[0, 0] = 0.0
    c.x[1, 0] = np.where(np.arange(128) % 2, 3e38, 1e30)          # the squares overflow, the norm does not
    c.x[2, 1] *= 1e-30                                            # the squares vanish beside eps
    q, k, _ = c.parts()
    qo, ko = P.qk_rope(c.rope(P), q, k, c.positions())
    _near(qo, *c.ref("q"), False)
    _near(ko, *c.ref("k"), False)
    c.x[0, 0, 5], c.x[3, 1, 9] = np.inf, np.nan
    q, k, _ = c.parts()
    qo, ko = P.qk_rope(c.rope(P), q, k, c.positions())
    y = _host(qo)
    assert np.isnan(y[0, 0]).any() and np.isnan(y[3, 1]).all() and np.isfinite(y[[0, 3], [1, 0]]).all()
    assert np.isfinite(y[1:3]).all() and np.isfinite(_host(ko)).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("eps", [2.0 ** -149, 2.0 ** -120, 1.5 * 2.0 ** 127])
def test_any_eps_and_any_size_of_values(P, D, eps):
    """Squares that vanish beside an eps that is as small, and sums over fp32's range.
    Results under its normal values round, five times at most (by the power, the gain, two
    products, a sum; gains are under 2), to multiples of 2^-149: up to 8 of them more."""
    sizes = (2.0 ** -148, 1e-40, 2.0 ** -75, 2.0 ** -70, 1e-10, 1e18, 3e38)
    c = Case(len(sizes), 3, 1, D, D, "f32")
    for t, size in enumerate(sizes):
        x = c.x[t].astype(np.float64)
        c.x[t] = x * (size / np.abs(x).max(-1, keepdims=True))
    c.x[1, 0], c.x[6, 1, 7] = 0.0, 1e-25
    assert np.abs(c.gq).max() < 2
    q, k, _ = c.parts()
    rope = P.Rope(_dev(c.inv), q_gain=_dev(c.gq), k_gain=_dev(c.gk), eps=eps)
    for y, x, g in zip(P.qk_rope(rope, q, k, c.positions()), (c.x[:, :3], c.x[:, 3:4]), (c.gq, c.gk), strict=True):
        ref, size = R.turned(x, g, eps, c.pos, c.inv, None, False)
        err, b = np.abs(_host(y) - ref), R.bound(ref, size, False) + 8 * 2.0 ** -149
        assert (err <= b).all(), (np.argwhere(err > b)[:4], err[err > b][:4], b[err > b][:4])


def test_a_side_without_heads(P):
    c = Case(5, 4, 2, 128, 128, "f32")
    q, k, _ = c.parts()
    rope, pos = c.rope(P), c.positions()
    both = P.qk_rope(rope, q, k, pos)
    assert (P.qk_rope(rope, q, k[:, :0], pos)[0] == both[0]).all()
    assert (P.qk_rope(rope, q[:, :0], k, pos)[1] == both[1]).all()


# ---- into the cache ------------------------------------------------------------------

def _rows(cache, slots):
    """Codes or values and scales of the slots: tokens x heads x ..."""
    s = slots.long()
    page, at = s // cache.page_tokens, s % cache.page_tokens
    pick = lambda t: None if t is None else t[page, :, at]  # noqa: E731
    return pick(cache.k), pick(cache.v), pick(cache.k_scale), pick(cache.v_scale)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_kv_append(P, case, act, kv):
    import torch

    c = Case(act=act, **case)
    q, k, v = c.parts()
    page = 5
    pages = c.T // page + 3
    slots = torch.randperm(pages * page, device="cuda")[:c.T].to(torch.int32)
    cache, other = (P.KVCache.empty(pages, c.Hkv, page, c.D, _torch(kv)) for _ in range(2))
    qo = P.kv_append(cache, c.rope(P), k, v, slots, c.positions(), q=q)
    _near(qo, *c.ref("q"), act == "bf16", "q")
    P.kv_write(other, k, v, slots)                       # the values are kv_write's, bit for bit
    gk, gv, ks, vs = _rows(cache, slots)
    _, wv, _, ws = _rows(other, slots)
    assert torch.equal(gv.view(torch.int8), wv.view(torch.int8)) and (kv == "bf16" or torch.equal(vs, ws))
    ref, size = c.ref("k")
    if kv == "bf16":
        _near(gk, ref, size, True, "k")
    else:
        err = np.abs(_host(gk) * _host(ks)[..., None] - ref)
        assert (err <= R.code_bound(ref, size)).all()
        assert int(gk.abs().max()) <= 127
    if act == "f32" and kv == "bf16":                    # one rounding, as in two calls
        P.kv_write(other, P.qk_rope(c.rope(P), q, k, c.positions())[1], v, slots)
        assert torch.equal(gk.view(torch.int16), _rows(other, slots)[0].view(torch.int16))


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_slots_outside_skip_and_nothing_else_is_written(P, kv):
    import torch

    c = Case(6, 4, 2, 64, 64, "f32")
    q, k, v = c.parts()
    slots = torch.tensor([3, -1, 40, 7, 2 ** 31 - 1, 11], dtype=torch.int32, device="cuda")
    cache = P.KVCache.empty(4, 2, 10, 64, _torch(kv))
    parts = [t for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
    for t in parts:
        t.fill_(77)
    qo = P.kv_append(cache, c.rope(P), k, v, slots, c.positions(), q=q)
    _near(qo, *c.ref("q"), False)                        # the queries of skipped tokens too
    rest = torch.ones(4, 10, dtype=torch.bool, device="cuda")
    for s in (3, 7, 11):
        rest[s // 10, s % 10] = False
    for t in parts:
        assert (t.transpose(1, 2)[rest] == 77).all()
    assert P.kv_append(cache, c.rope(P), k, v, slots, c.positions()) is None


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_codes_are_kv_writes_where_rounding_is_close(P, act):
    """Halves, zeros, rows of few bits and of the smallest values: the same codes and scales, bit for bit."""
    import torch

    rng = np.random.default_rng(44)
    T, Hkv, D = 400, 3, 64
    v = rng.standard_normal((T, Hkv, D)).astype(np.float32)
    v[:100] = (rng.integers(-254, 255, (100, Hkv, D)) / 2).astype(np.float32)        # halves of a scale of 1
    v[:100, :, 0] = 127.0
    v[100:150] = (rng.integers(-300, 300, (50, Hkv, D)) * 2.0 ** -149).astype(np.float32)
    v[150:160] = 0.0
    v[160:200] *= 2.0 ** rng.integers(-120, 120, (40, 1, 1)).astype(np.float32)
    v[200:300] = rng.integers(-127, 128, (100, Hkv, D)) * np.float32(0.1)              # near whole codes
    vd = _dev(v, act)
    k = torch.randn(T, Hkv, D, device="cuda").to(_torch(act))
    slots = torch.randperm(T + 8, device="cuda")[:T].to(torch.int32)
    one, two = (P.KVCache.empty(T + 8, Hkv, 1, D, torch.int8) for _ in range(2))
    rope = P.Rope(torch.zeros(0, device="cuda"))                                       # neither norm nor rotation
    P.kv_append(one, rope, k, vd, slots, torch.zeros(T, dtype=torch.int32, device="cuda"))
    P.kv_write(two, k, vd, slots)
    for a, b in zip(_rows(one, slots), _rows(two, slots)):
        assert torch.equal(a, b)


def test_non_finite_rows_have_nan_scales(P):
    import torch

    c = Case(3, 2, 2, 64, 64, "f32", norm="")
    c.x[1, 2, 7] = np.inf
    c.x[2, 5, 0] = np.nan
    q, k, v = c.parts()
    cache = P.KVCache.empty(1, 2, 4, 64, torch.int8)
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    P.kv_append(cache, c.rope(P), k, v, slots, c.positions())
    _, _, ks, vs = _rows(cache, slots)
    bad = torch.zeros(3, 2, dtype=torch.bool, device="cuda")
    bad[1, 0] = True
    assert torch.equal(torch.isnan(ks), bad)
    bad[1, 0], bad[2, 1] = False, True
    assert torch.equal(torch.isnan(vs), bad)


def test_a_step_in_a_graph_follows_its_inputs(P):
    """Positions, slots and rows of a captured step are read when it is replayed."""
    import torch

    c = Case(4, 4, 2, 128, 128, "f32")
    x = _dev(c.x)
    q, k, v = x.split((4, 2, 2), 1)
    cache, rope, pos = P.KVCache.empty(3, 2, 8, 128, torch.int8), c.rope(P), c.positions()
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    qo = torch.empty(4, 4, 128, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        P.kv_append(cache, rope, k, v, slots, pos, q=q, q_out=qo)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.kv_append(cache, rope, k, v, slots, pos, q=q, q_out=qo)
    for seed in (1, 2):
        d = Case(4, 4, 2, 128, 128, "f32", seed=seed)
        d.gq, d.gk = c.gq, c.gk
        x.copy_(_dev(d.x))
        pos.copy_(d.positions())
        slots.copy_(torch.arange(4, device="cuda") + 4 * seed)
        g.replay()
        torch.cuda.synchronize()
        _near(qo, *d.ref("q"), False)
        gk, _, ks, _ = _rows(cache, slots)
        ref, size = d.ref("k")
        assert (np.abs(_host(gk) * _host(ks)[..., None] - ref) <= R.code_bound(ref, size)).all()


def test_a_side_stream(P):
    import torch

    c = Case(64, 8, 2, 128, 128, "bf16")
    q, k, _ = c.parts()
    rope, pos = c.rope(P), c.positions()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    qo, ko = P.qk_rope(rope, q, k, pos, stream=s)
    s.synchronize()
    _near(qo, *c.ref("q"), True)
    _near(ko, *c.ref("k"), True)


def test_rows_past_32_bits_of_offset(P):
    """Tokens so far apart that their offsets pass 2^31 values."""
    import torch

    c = Case(3, 1, 1, 64, 64, "bf16", norm="")
    stride = 2 ** 30 + 8
    big = torch.empty(2 * stride + 3 * 64, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((3, 3, 64), (stride, 64, 1))
    x.copy_(_dev(c.x, "bf16"))
    q, k, _ = x.split((1, 1, 1), 1)
    qo, ko = P.qk_rope(c.rope(P), q, k, c.positions())
    _near(qo, *c.ref("q"), True)
    P.qk_rope(c.rope(P), q, k, c.positions(), q_out=q, k_out=k)
    _near(q, *c.ref("q"), True)
    _near(k, *c.ref("k"), True)
