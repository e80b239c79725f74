"""The edges of the paged cache and the attention operators: rows of the
smallest subnormals, value scales that differ by orders of magnitude."""
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


def _decode_weighted(P, k, v, q, act, page, width, what):
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
    out = _host(P.attn_decode(qd, cache, table, lens))[0]
    (kc, ks), (vc, vs) = R.quantise(k), R.quantise(v)
    kk, vv = (c.astype(np.float64) * s[:, None].astype(np.float64) for c, s in ((kc, ks), (vc, vs)))
    for h in range(len(q)):
        ref, bound = _weighted_bound(q[h], kk, vv, vs, D ** -0.5, act == "bf16")
        err = np.abs(out[h] - ref)
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
