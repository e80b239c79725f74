"""The edges of the paged cache and the attention operators: rows of the
smallest subnormals, value scales that differ by orders of magnitude, buffers on
other streams, thousands of prompts, values that are not finite."""
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


def _host(t):
    return t.double().cpu().numpy()


# ---- the cache -------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128, 256])
def test_codes_of_subnormal_rows_stay_in_range(P, D):
    """Under a maximum of some 2^-135 the scale max / 127 is a subnormal of few
    bits, and the quotients pass 127: the codes stop there."""
    import torch

    unit = 2.0 ** -149
    tops = [1, 63, 64, 127, 128, 190, 191, 255, 318, 5000, 70001, 2 ** 20 + 1, 2 ** 23 - 1, 2 ** 23, 2 ** 24]
    rng = np.random.default_rng(D)
    x = np.zeros((2 * len(tops), 1, D), np.float32)
    for i, top in enumerate(tops):
        x[2 * i:2 * i + 2, 0] = rng.integers(-top, top + 1, D) * unit
        x[2 * i, 0, 5], x[2 * i + 1, 0, D - 1] = top * unit, -top * unit
    xd = torch.from_numpy(x).cuda()
    cache = P.KVCache.empty(len(x), 1, 1, D, torch.int8)
    slots = torch.arange(len(x), dtype=torch.int32, device="cuda")
    P.kv_write(cache, xd, -xd, slots)
    s = np.abs(x).max(-1) / np.float32(127)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s[..., None] > 0, np.clip(np.rint(x / s[..., None]), -127, 127), 0).astype(np.int8)
    assert (np.abs(c) == 127).any() and (s == 0).any()
    np.testing.assert_array_equal(cache.k_scale.cpu().numpy()[:, 0], s)
    np.testing.assert_array_equal(cache.k.cpu().numpy()[:, 0], c)
    np.testing.assert_array_equal(cache.v.cpu().numpy()[:, 0], -c)
    k, v = P.kv_read(cache, slots, dtype=torch.float32)
    np.testing.assert_array_equal(k.cpu().numpy(), c * s[..., None])
    np.testing.assert_array_equal(v.cpu().numpy(), -c * s[..., None])


# ---- decode over int8: weights and value scales ------------------------------------

def _weighted_bound(q, k, v, vs, scale, bf16_out):
    """The definition's output in 64 bits and what it may be off by, for one query
    row over keys k, values v (rows as stored, their scales vs).

    A score's error is that of attn_ref, for each key by itself: eps_j = 2^-21
    sqrt(D) scale sum_d |q_d k_jd| + 2^-20.  It changes the normalised weight p_j by
    at most p_j (eps_j + sum_i p_i eps_i) to first order (a tenth more covers the
    rest).  Weights and sums are fp32 or a pair of fp16 terms, 2^-21 of each
    product and 2^-24 of the sum for each addition; a pair of terms under the 16-bit
    range keeps 2^-35 of the largest weighted scale, doubled for the power of two
    above it, times a code of at most 127: 2^-27 for each key."""
    q, k, v, vs = (np.asarray(a, np.float64) for a in (q, k, v, vs))
    s = scale * (k @ q)
    p = np.exp(s - s.max())
    p /= p.sum()
    out = p @ v
    eps = 2.0 ** -21 * np.sqrt(len(q)) * scale * (np.abs(k) @ np.abs(q)) + 2.0 ** -20
    bound = 1.1 * (p * (eps + p @ eps)) @ np.abs(v)
    bound = bound + (2.0 ** -21 + len(k) * 2.0 ** -24) * (p @ np.abs(v)) + len(k) * 2.0 ** -27 * (p * vs).max()
    return out, bound + (2.0 ** -8 * np.abs(out) if bf16_out else 0)


def _decode_weighted(P, k, v, q, act, page, width, what, copies=1):
    """One sequence, or `copies` of it over the same pages (a CTA then takes whole ones)."""
    import torch

    n, D = len(k), k.shape[-1]
    pages = -(-n // page)
    cache = P.KVCache.empty(pages, 1, page, D, torch.int8)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()
    P.kv_write(cache, dev(k)[:, None], dev(v)[:, None], slots)
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, :pages] = torch.arange(pages, dtype=torch.int32)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = R.bf16(q) if act == "bf16" else q.astype(np.float32)
    qd = dev(q)[None].to(torch.bfloat16 if act == "bf16" else torch.float32)
    out = P.attn_decode(qd.repeat(copies, 1, 1), cache, table.repeat(copies, 1), lens.repeat(copies))
    out = _host(out[[0, copies // 2, copies - 1]])
    (kc, ks), (vc, vs) = R.quantise(k), R.quantise(v)
    kk, vv = (c.astype(np.float64) * s[:, None].astype(np.float64) for c, s in ((kc, ks), (vc, vs)))
    for h in range(len(q)):
        ref, bound = _weighted_bound(q[h], kk, vv, vs, D ** -0.5, act == "bf16")
        err = np.abs(out[:, h] - ref)
        assert (err <= bound).all(), f"{what} head {h}: off by {(err / bound).max():.3g} of the bound"


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 5), (128, 12), (256, 3)])
@pytest.mark.parametrize("width", [40, 200])      # a cluster's call, and runs
def test_a_loud_value_of_no_weight_costs_no_accuracy(P, act, D, G, width):
    rng = np.random.default_rng([D, G])
    n = 300
    for r in (8, 16, 24, 32, 60):
        for where in (0, 17, 150, n - 1):
            base = rng.standard_normal(D)
            q = base + 0.05 * rng.standard_normal((G, D))
            k, v = 0.3 * rng.standard_normal((n, D)), rng.standard_normal((n, D))
            # weight 2^-r e^-25 or so: a score that much under the others'
            k[where] = -base * (r * np.log(2) + 25) * np.sqrt(D) / (base @ base)
            v[where] *= 2.0 ** r
            _decode_weighted(P, k.astype(np.float32), v.astype(np.float32), q, act, 16, width, f"2^{r} at {where}")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-35, 1e-30, 1e30])
def test_values_of_any_size(P, act, size):
    rng = np.random.default_rng(3)
    n, D = 150, 128
    k, v = 0.3 * rng.standard_normal((n, D)), size * rng.uniform(0.5, 2.0, (n, D))
    q = rng.standard_normal((5, D))
    for width in (40, 200):
        _decode_weighted(P, k.astype(np.float32), v.astype(np.float32), q, act, 16, width, f"{size}")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 5), (128, 12), (256, 3)])
def test_a_great_value_before_scores_that_leave_it_no_weight(P, act, D, G):
    """The weights so far underflow at once, and the values that follow are smaller
    by more than fp32's exponents (2^140)."""
    rng = np.random.default_rng([D, G, 1])
    n = 300
    base = rng.standard_normal(D)
    q = base + 0.05 * rng.standard_normal((G, D))
    k, v = 0.05 * rng.standard_normal((n, D)), rng.standard_normal((n, D)) * 2.0 ** -70
    k[n // 2:] += base * 150 * np.sqrt(D) / (base @ base)
    v[:n // 2] *= 2.0 ** 140
    for width in (40, 200):
        for copies in (1, 400):
            _decode_weighted(P, k.astype(np.float32), v.astype(np.float32), q, act, 16, width, "2^140", copies)


# ---- streams -----------------------------------------------------------------------

def test_default_buffers_on_another_stream(P):
    """Calls queued on a stream behind other work, with the buffers they allocate
    themselves, while the current stream fills new tensors of the same sizes."""
    import torch

    rng = np.random.default_rng(51)
    B, Hkv, G, D, page = 5, 4, 5, 128, 16
    lens = [3000, 1, 777, 2048, 90]
    pages = -(-max(lens) // page)
    cache = P.KVCache.empty(B * pages, Hkv, page, D, torch.int8)
    table = torch.randperm(B * pages, device="cuda").to(torch.int32).view(B, pages)
    slots = torch.arange(B * pages * page, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(len(slots), Hkv, D, device="cuda") for _ in range(2))
    q = torch.randn(B, Hkv * G, D, device="cuda")
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # few queries over many keys: the prompts' keys are cut into parts
    nq, nk = 40, 9000
    pq, pk, pv = (torch.randn(n, h, D, device="cuda").bfloat16() for n, h in ((nq, G), (nk, 1), (nk, 1)))
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (nq, nk))
    assert P.attn_prefill_workspace_bytes(1, nq, nk, G, 1, D, P.PTQ_BF16) > 0

    def calls(stream):
        kr, vr = P.kv_read(cache, slots[:999], dtype=torch.float32, stream=stream)
        return [kr, vr, P.attn_decode(q, cache, table, lens_d, stream=stream),
                P.attn_prefill(pq, pk, pv, cu_q, cu_k, stream=stream)]

    P.kv_write(cache, k, v, slots)
    want = [t.clone() for t in calls(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)   # some 10 ms
        got = calls(side)
        sizes = [P.attn_decode_workspace_bytes(B, Hkv * G, Hkv, D, P.PTQ_F32),
                 P.attn_prefill_workspace_bytes(1, nq, nk, G, 1, D, P.PTQ_BF16)] + [t.nbytes for t in got]
        fill = [torch.full((n,), 0xAA, dtype=torch.uint8, device="cuda") for n in sizes * 2]
        torch.cuda.current_stream().synchronize()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert all((t == 0xAA).all() for t in fill)
        del got, fill


def test_default_buffers_in_a_graph_of_two_streams(P):
    import torch

    torch.manual_seed(5)
    q, k, v = (torch.randn(n, h, 128, device="cuda").bfloat16() for n, h in ((40, 5), (9000, 1), (9000, 1)))
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (40, 9000))
    want = P.attn_prefill(q, k, v, cu_q, cu_k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    P.attn_prefill(q, k, v, cu_q, cu_k, stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one = P.attn_prefill(q, k, v, cu_q, cu_k)
        side.wait_stream(torch.cuda.current_stream())
        two = P.attn_prefill(q, k, v, cu_q, cu_k, stream=side)
        three = P.attn_prefill(q, k, v, cu_q, cu_k)
        torch.cuda.current_stream().wait_stream(side)
    for t in (one, two, three):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in (one, two, three))


# ---- prompts: many sequences ---------------------------------------------------------

def _prompts(P, rng, nqs, nks, Hkv, G, D, causal, pick):
    """Packed prompts against the definition, the sequences `pick` of them."""
    import torch

    q, k, v = (R.bf16(rng.standard_normal((n, h, D)).astype(np.float32))
               for n, h in ((sum(nqs), Hkv * G), (sum(nks), Hkv), (sum(nks), Hkv)))
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(n)]) for n in (nqs, nks))
    dev = lambda x: torch.from_numpy(x).cuda()
    lse = torch.full((sum(nqs), Hkv * G), 7.0, device="cuda")
    out = P.attn_prefill(dev(q).bfloat16(), dev(k).bfloat16(), dev(v).bfloat16(), dev(cu_q.astype(np.int32)),
                         dev(cu_k.astype(np.int32)), causal=causal, lse=lse)
    P.device_check()
    out, lse = _host(out), _host(lse)
    assert np.isfinite(out).all()
    for b in pick:
        (q0, q1), (k0, k1) = cu_q[b:b + 2], cu_k[b:b + 2]
        i, j = np.arange(q1 - q0)[:, None], np.arange(k1 - k0)[None]
        seen = (j <= i + (k1 - k0) - (q1 - q0)) if causal else np.ones((q1 - q0, k1 - k0), bool)
        rows = np.arange(q1 - q0) if q1 - q0 < 200 else np.unique(np.linspace(0, q1 - q0 - 1, 60).astype(int))
        for hq in range(Hkv * G):
            ref = R.attend(q[q0 + rows, hq], k[k0:k1, hq // G], v[k0:k1, hq // G], D ** -0.5, seen[rows])
            R.check(out[q0 + rows, hq], lse[q0 + rows, hq], ref, True, True, f"seq {b} head {hq}")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,long,D,Hkv,G", [(33, 200, 128, 1, 5), (65, 900, 256, 1, 2), (700, 900, 64, 2, 1),
                                            (3001, 700, 64, 1, 2), (20000, 3000, 64, 1, 1), (140001, 3000, 64, 1, 1)])
def test_many_prompts(P, B, long, D, Hkv, G, causal):
    """More sequences than one step of the planning warp sees, most of them short;
    in the large batches several runs of a long prompt are dealt out at once."""
    rng = np.random.default_rng([B, D])
    nqs = rng.integers(0, 4, B)
    at = [0, B // 3, B // 2, B - 2]
    nqs[at] = [long, long // 2, 130, long - 77]
    nks = nqs + (rng.random(B) < 0.3) * rng.integers(0, 3, B)
    pick = list(range(min(B, 40))) + at + list(range(max(0, B - 40), B)) + list(rng.integers(0, B, 60))
    _prompts(P, rng, nqs.tolist(), nks.tolist(), Hkv, G, D, causal, sorted(set(pick)))


def test_planning_grows_with_the_batch_alone(P):
    """65,536 prompts of a token: the planning warp's walk once took a step for
    every 32 sequences for every item (3.5 million of them a CTA, a third of a
    second); 3,450 items a CTA take some milliseconds."""
    import torch

    n, H, D = 65536, 8, 64
    q, k, v = (torch.randn(n, H, D, device="cuda").bfloat16() for _ in range(3))
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    out = P.attn_prefill(q, k, v, cu, cu)
    P.device_check()
    assert torch.equal(out, v)              # one key has all the weight
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    P.attn_prefill(q, k, v, cu, cu, out=out)
    b.record()
    torch.cuda.synchronize()
    assert a.elapsed_time(b) < 60
    print(f"{a.elapsed_time(b):.2f} ms")


# ---- prompts: values that are not finite -----------------------------------------------

def _timed(call):
    import torch

    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    call()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


class Long:
    """Random queries, keys and values of some prompts, their clean outputs, and the
    outputs and time with other values."""

    def __init__(self, P, seed, nqs, nks, Hkv, G, D, causal=True):
        import torch

        torch.manual_seed(seed)
        self.P, self.D, self.G, self.causal = P, D, G, causal
        self.q, self.k, self.v = (torch.randn(n, h, D, device="cuda").bfloat16()
                                  for n, h in ((sum(nqs), Hkv * G), (sum(nks), Hkv), (sum(nks), Hkv)))
        self.cu = [torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
                   for n in (nqs, nks)]
        self.run(self.v)
        self.clean, self.lse, self.ms = self.run(self.v)

    def run(self, v):
        import torch

        out, lse = torch.empty_like(self.q), torch.empty(self.q.shape[:2], device="cuda")
        ms = _timed(lambda: self.P.attn_prefill(self.q, self.k, v, *self.cu, causal=self.causal, out=out, lse=lse))
        self.P.device_check()
        return out, lse, ms

    def check_row(self, out, lse, i, hq, v, keys):
        """Query i of all, head hq, over `keys`."""
        h = hq // self.G
        ref = R.attend(_host(self.q[i, hq])[None], _host(self.k[keys, h]), _host(v[keys, h]), self.D ** -0.5)
        R.check(_host(out[i, hq])[None], _host(lse[i, hq])[None], ref, True, True, f"query {i} head {hq}")


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("D,Hkv,G", [(128, 2, 5), (64, 2, 4), (256, 1, 6)])
def test_a_value_seen_by_all_spoils_its_column_alone(P, D, Hkv, G, bad):
    """The first token's value not finite: the long prompt's rows are as without it
    but for one column, and none is computed again one by one (which took
    hundreds of times the prompt's own time)."""
    import torch

    s = Long(P, D, [8192], [8192], Hkv, G, D)
    v = s.v.clone()
    v[0, 0, 7] = bad
    out, lse, ms = s.run(v)
    assert torch.equal(lse, s.lse)
    assert (torch.isnan(out[:, :G, 7]) if bad != bad else torch.isposinf(out[:, :G, 7])).all()
    out[:, :G, 7] = s.clean[:, :G, 7]
    assert torch.equal(out, s.clean)
    assert ms < 5 * s.ms + 0.5, (ms, s.ms)


@pytest.mark.parametrize("where", [8191, 8000, 4100])
@pytest.mark.parametrize("D,Hkv,G", [(128, 2, 5), (64, 2, 4), (256, 1, 6)])
def test_a_hidden_value_reaches_no_row(P, D, Hkv, G, where):
    """Rows before the token are as without it, to the last bit or (those whose tile
    it spoils) to the definition; the time stays near the prompt's."""
    import torch

    s = Long(P, D, [8192], [8192], Hkv, G, D)
    v = s.v.clone()
    v[where, 0] = float("nan")
    out, lse, ms = s.run(v)
    assert torch.equal(lse, s.lse) and torch.equal(out[:, G:], s.clean[:, G:])
    assert torch.isnan(out[where:, :G]).all()
    moved = (out[:where, :G] != s.clean[:where, :G]).any(-1).nonzero().cpu().numpy()
    print(f"{len(moved)} rows differ, {ms:.2f} ms for {s.ms:.2f}")
    assert len(moved) == 0 or moved[:, 0].min() >= where - 512
    for i, hq in moved[:: max(1, len(moved) // 40)]:
        s.check_row(out, lse, i, hq, v, slice(0, i + 1))
    assert ms < 60


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,Hkv,G", [(128, 2, 5), (64, 2, 4), (256, 1, 6)])
def test_the_next_prompts_values_reach_no_row(P, D, Hkv, G, causal):
    """A prompt of NaN values after one whose last tile they share."""
    import torch

    for n in (4001, 4032, 4095):
        s = Long(P, D, [n, 300], [n, 300], Hkv, G, D, causal)
        v = s.v.clone()
        v[n:] = float("nan")
        out, lse, ms = s.run(v)
        assert torch.equal(out[:n], s.clean[:n]) and torch.equal(lse, s.lse)
        assert torch.isnan(out[n:]).all()
        assert ms < 3 * s.ms + 0.5, (ms, s.ms)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,Hkv,G", [(128, 2, 5), (64, 2, 4), (256, 1, 6)])
def test_a_short_prompts_neighbours_values_reach_no_row(P, D, Hkv, G, causal):
    import torch

    for n in (3, 130, 700, 1024, 1025, 1100):
        s = Long(P, D, [50, n, 40], [50, n, 40], Hkv, G, D, causal)
        v = s.v.clone()
        v[:50], v[50 + n:] = float("inf"), float("nan")
        out, lse, ms = s.run(v)
        assert torch.equal(lse, s.lse) and torch.isnan(out[50 + n:]).all()
        mine, clean = out[50:50 + n], s.clean[50:50 + n]
        moved = (mine != clean).any(-1).nonzero().cpu().numpy()
        for i, hq in moved[:: max(1, len(moved) // 25)]:
            s.check_row(out, lse, 50 + i, hq, s.v, slice(50, 50 + (i + 1 if causal else n)))
        assert torch.isfinite(mine).all() and (mine - clean).abs().max() < 0.1
        assert ms < 30


@pytest.mark.parametrize("D,G,nq,nk", [(128, 5, 40, 9000), (64, 1, 70, 12345), (256, 6, 9, 5000)])
def test_non_finite_values_where_the_keys_are_cut_into_parts(P, D, G, nq, nk):
    import torch

    assert P.attn_prefill_workspace_bytes(1, nq, nk, G, 1, D, P.PTQ_BF16) > 0
    s = Long(P, D, [nq], [nk], 1, G, D)
    v = s.v.clone()
    v[nk - 2, 0, 3] = float("nan")          # hidden from all but two queries
    v[100, 0, 5] = float("inf")             # seen by all
    out, lse, ms = s.run(v)
    assert torch.equal(lse[nq - 2:], s.lse[nq - 2:]) and torch.isposinf(out[..., 5]).all()
    assert torch.isnan(out[nq - 2:, :, 3]).all()
    keep = [d for d in range(D) if d != 5]
    assert torch.isfinite(out[:nq - 2, :, keep]).all()
    out[..., 5], v[100, 0, 5] = s.clean[..., 5], s.v[100, 0, 5]
    for i in range(0, nq - 2, max(1, nq // 5)):
        for hq in range(G):
            s.check_row(out, lse, i, hq, v, slice(0, i + nk - nq + 1))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_values_under_a_maximum_that_grows_a_little(P, D):
    """Weights may be 2^8 times the largest key's while they are summed, and the sums
    of values near 1e36 then overflow (147 x 132 x 1e36); relative to the largest key
    (132 x 1e36) they do not."""
    import torch

    n, nq = 260, 5
    q = torch.zeros(nq, 1, D, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(n, 1, D, device="cuda", dtype=torch.bfloat16)
    q[:, 0, 0], k[128:, 0, 0] = 1.0, 5.0     # scores of 0, then of 5 (7.2 in units of log2)
    v = (torch.rand(n, 1, D, device="cuda") + 0.5).mul(1e36).bfloat16()
    cu_q, cu_k = (torch.tensor([0, m], dtype=torch.int32, device="cuda") for m in (nq, n))
    out = P.attn_prefill(q, k, v, cu_q, cu_k, scale=1.0)
    for i in range(nq):
        ref = R.attend(_host(q[i]), _host(k[:n - nq + i + 1, 0]), _host(v[:n - nq + i + 1, 0]), 1.0)
        R.check(_host(out[i]), None, ref, True, True)


@pytest.mark.parametrize("D,Hkv,G", [(128, 2, 5), (64, 2, 4), (256, 1, 6)])
def test_strided_tensors_and_an_output_of_16_byte_alignment(P, D, Hkv, G):
    """Columns of one projection's rows, hidden and seen values that are not finite,
    an output 16 bytes off a 32-byte boundary: as with tensors of their own."""
    import torch

    nqs = [1300, 70, 5]
    s = Long(P, 9, nqs, nqs, Hkv, G, D)
    v = s.v.clone()
    v[1250, 0], v[1299], v[1305, 0, 2], v[40, Hkv - 1, 1] = float("nan"), float("inf"), float("nan"), float("inf")
    want, lse, _ = s.run(v)
    row = torch.cat([s.q, s.k, v], 1)
    n, Hq = s.q.shape[:2]
    buf = torch.full((n * Hq * D + 24,), 9.0, device="cuda", dtype=torch.bfloat16)
    out = buf[8:-16].view(n, Hq, D)
    assert out.data_ptr() % 32 == 16
    lse2 = torch.empty_like(lse)
    P.attn_prefill(row[:, :Hq], row[:, Hq:Hq + Hkv], row[:, Hq + Hkv:], *s.cu, out=out, lse=lse2)
    assert torch.equal(lse, lse2) and torch.equal(out.nan_to_num(7.0), want.nan_to_num(7.0))
    assert torch.equal(out.isnan(), want.isnan()) and (buf[:8] == 9).all() and (buf[-16:] == 9).all()
