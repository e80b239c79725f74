"""Attention of packed prompts on the GPU, against plain 64-bit arithmetic
(tests/attn_ref.py)."""
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


def _dev(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(torch.bfloat16)


def _host(t):
    return t.double().cpu().numpy()


def _cu(lens):
    import torch

    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _values(rng, shape):
    return R.bf16(rng.standard_normal(shape).astype(np.float32))


def _seen(nq, nk, causal):
    i, j = np.arange(nq)[:, None], np.arange(nk)[None]
    return (j <= i + nk - nq) if causal else np.ones((nq, nk), bool)


def _check(q, k, v, out, lse, nqs, nks, Hkv, scale, causal, what="", rows=None):
    """rows: which queries of each sequence are checked (all when None)."""
    G = q.shape[1] // Hkv
    aq = ak = 0
    for b, (nq, nk) in enumerate(zip(nqs, nks)):
        pick = np.arange(nq) if rows is None else np.unique(np.clip(rows, 0, nq - 1)) if nq else np.arange(0)
        seen = _seen(nq, nk, causal)[pick]
        for hq in range(q.shape[1]):
            h = hq // G
            ref = R.attend(q[aq + pick, hq], k[ak:ak + nk, h], v[ak:ak + nk, h], scale, seen)
            R.check(out[aq + pick, hq], lse[aq + pick, hq], ref, True, True, f"{what} seq {b} head {hq}")
        aq, ak = aq + nq, ak + nk


def _case(P, seed, nqs, nks, Hkv, G, D, causal, scale=None, rows=None):
    import torch

    rng = np.random.default_rng(seed)
    q, k, v = (_values(rng, (n, h, D)) for n, h in ((sum(nqs), Hkv * G), (sum(nks), Hkv), (sum(nks), Hkv)))
    lse = torch.full((sum(nqs), Hkv * G), 7.0, device="cuda")
    out = P.attn_prefill(_dev(q), _dev(k), _dev(v), _cu(nqs), _cu(nks), causal=causal, scale=scale, lse=lse)
    _check(q, k, v, _host(out), _host(lse), nqs, nks, Hkv, scale or D ** -0.5, causal, rows=rows)


HEADS = [(64, 2, 1), (128, 2, 5), (256, 1, 6), (128, 1, 8), (64, 1, 20), (256, 1, 3), (128, 1, 16), (64, 1, 7)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,Hkv,G", HEADS)
def test_packed_prompts(P, D, Hkv, G, causal):
    # lengths of zero and one, around the tiles' sizes, ragged
    nqs = [1, 0, 2, 64, 17, 128, 0, 129, 200, 1]
    _case(P, [D, G], nqs, nqs, Hkv, G, D, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,Hkv,G", [(64, 1, 1), (128, 1, 5), (256, 1, 6)])
def test_prefixes_and_rows_without_keys(P, D, Hkv, G, causal):
    # more keys than queries, fewer (the first queries then see none under the
    # causal mask), none at all
    nqs = [1, 5, 130, 300, 40, 128, 9, 260]
    nks = [300, 133, 129, 20, 0, 256, 640, 3]
    _case(P, [D, G, 2], nqs, nks, Hkv, G, D, causal)


@pytest.mark.parametrize("D,Hkv,G,n", [(128, 1, 1, 1537), (128, 1, 5, 700), (64, 2, 2, 1100), (256, 1, 2, 1000)])
def test_longer_prompts(P, D, Hkv, G, n):
    rows = np.concatenate([np.arange(0, n, 61), [127, 128, 255, 256, 511, 512, n - 2, n - 1]])
    _case(P, [n], [n], [n], Hkv, G, D, True, rows=rows)


@pytest.mark.parametrize("D,G,nq,nk", [(128, 5, 3, 9000), (256, 6, 1, 5000), (64, 1, 40, 12345)])
def test_few_queries_over_a_long_prefix(P, D, G, nq, nk):
    _case(P, [nq, nk], [nq, 2], [nk, 300], 1, G, D, True)


def test_scale_and_large_scores(P):
    _case(P, 5, [150, 33], [150, 60], 1, 2, 128, True, scale=1.75)


def test_strides_stream_and_guards(P):
    # q, k and v as columns of one fused projection's output, a stream of its
    # own, out inside a guarded buffer
    import torch

    rng = np.random.default_rng(20)
    n, Hkv, G, D = 190, 2, 3, 128
    x = _values(rng, (n, Hkv * G + 2 * Hkv, D))
    xd = _dev(x)
    Hq = Hkv * G
    buf = torch.full((n * Hq * D + 4096,), 9.0, dtype=torch.bfloat16, device="cuda")
    out, lse = buf[2048:-2048].view(n, Hq, D), torch.empty(n, Hq, device="cuda")
    cu = _cu([100, 90])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    P.attn_prefill(xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], cu, cu, out=out, lse=lse, stream=side)
    side.synchronize()
    _check(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], _host(out), _host(lse), [100, 90], [100, 90], Hkv,
           D ** -0.5, True)
    assert (buf[:2048] == 9).all() and (buf[-2048:] == 9).all()


def test_rows_of_no_sequence_and_offsets_out_of_range(P):
    import torch

    rng = np.random.default_rng(21)
    q, k, v = (_values(rng, (80, h, 64)) for h in (2, 1, 1))
    out, lse = torch.full((80, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda"), torch.zeros(80, 2, device="cuda")
    cu = torch.tensor([10, 40, 70], dtype=torch.int32, device="cuda")
    P.attn_prefill(_dev(q), _dev(k), _dev(v), cu, cu, out=out, lse=lse)
    assert (out[:10] == 3).all() and (out[70:] == 3).all() and (lse[:10] == 0).all()
    _check(q[10:70], k[10:70], v[10:70], _host(out)[10:70], _host(lse)[10:70], [30, 30], [30, 30], 1, 0.125, True)
    wild = torch.tensor([-9, 50, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    P.attn_prefill(_dev(q), _dev(k), _dev(v), wild, wild, out=out, lse=lse)
    _check(q, k, v, _host(out), _host(lse), [50, 30], [50, 30], 1, 0.125, True)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 5), (256, 2)])
def test_non_finite_keys_and_values_reach_only_the_queries_that_see_them(P, bad, D, G):
    import torch

    rng = np.random.default_rng(22)
    nqs, nks = [150, 140], [150, 200]
    q, k, v = (_values(rng, (n, h, D)) for n, h in ((290, G), (350, 1), (350, 1)))
    k2, v2 = k.copy(), v.copy()
    v2[70, 0, 3], k2[200, 0, 5], v2[150, 0, 0] = bad, np.nan, bad   # tokens 70 | 50 and 0 of the two sequences
    lse = torch.empty(290, G, device="cuda")
    out = P.attn_prefill(_dev(q), _dev(k2), _dev(v2), _cu(nqs), _cu(nks), lse=lse)
    got, l = _host(out), _host(lse)
    # sequence 0: queries before token 70 are untouched by it, those after it
    # see it in dimension 3 alone
    clean = [np.delete(x, 3, -1) for x in (got[:150],)][0]
    ok = np.isfinite(clean).all()
    assert ok and not np.isfinite(got[70:150, :, 3]).any()
    for h in range(G):
        ref = R.attend(q[:70, h], k[:150, 0], v[:150, 0], D ** -0.5, _seen(150, 150, True)[:70])
        R.check(got[:70, h], l[:70, h], ref, True, True)
    # sequence 1 (60 keys before its queries): token 0 in dimension 0 for all,
    # the NaN key 50 is seen by all
    assert np.isnan(got[150:]).all() and np.isnan(l[150:]).all()


def test_reproducible_and_capturable(P):
    import torch

    rng = np.random.default_rng(23)
    nqs = [300, 1, 513, 40]
    n = sum(nqs)
    q, k, v = (_dev(_values(rng, (n, h, 128))) for h in (10, 2, 2))
    cu = _cu(nqs)
    need = P.attn_prefill_workspace_bytes(4, n, n, 10, 2, 128, P.PTQ_BF16)
    ws = torch.full((max(1, need),), 0xff, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(n, 10, device="cuda")

    def call():
        P.attn_prefill(q, k, v, cu, cu, out=out, lse=lse, workspace=ws)

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
    cu.copy_(_cu([10, 500, 0, n - 510]))
    g.replay()
    again = out.clone()
    call()
    assert torch.equal(out, again) and not torch.equal(out, first)


def test_prompt_then_decode_agree(P):
    # the last query of a prompt equals the decode of that token over a bf16
    # cache of the same keys and values
    import torch

    rng = np.random.default_rng(24)
    n, Hkv, G, D = 333, 2, 4, 128
    q, k, v = (_dev(_values(rng, (n, h, D))) for h in (Hkv * G, Hkv, Hkv))
    out = P.attn_prefill(q, k, v, _cu([n]), _cu([n]))
    cache = P.KVCache.empty(22, Hkv, 16, D, torch.bfloat16)
    table = torch.randperm(22, device="cuda")[:21].to(torch.int32)[None]
    j = torch.arange(n, device="cuda")
    slots = (table[0, j // 16] * 16 + j % 16).to(torch.int32)
    P.kv_write(cache, k, v, slots)
    one = P.attn_decode(q[-1:], cache, table.contiguous(), torch.tensor([n], dtype=torch.int32, device="cuda"))
    top = v.abs().max().item()
    d = (one.double() - out[-1:].double()).abs()
    assert (d <= 2 * 2.0 ** -8 * one.double().abs() + 2.0 ** -9 * top + 1e-4 * top).all()


def test_refusals(P):
    import torch

    q, k = torch.zeros(4, 4, 128, device="cuda"), torch.zeros(4, 2, 128, device="cuda")
    with pytest.raises(P.PTQError, match="UNSUPPORTED"):
        P.attn_prefill(q, k, k, _cu([4]), _cu([4]))
    q, k = q.bfloat16(), k.bfloat16()
    with pytest.raises(ValueError, match="contiguous"):
        P.attn_prefill(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, _cu([4]), _cu([4]))
    with pytest.raises(TypeError, match="int32"):
        P.attn_prefill(q, k, k, _cu([4]).long(), _cu([4]))
    with pytest.raises(P.PTQError, match="SHAPE"):
        P.attn_prefill(q, torch.zeros(4, 3, 128, device="cuda", dtype=torch.bfloat16), torch.zeros(
            4, 3, 128, device="cuda", dtype=torch.bfloat16), _cu([4]), _cu([4]))
    with pytest.raises(P.PTQError, match="VALUE"):
        P.attn_prefill(q, k, k, _cu([4]), _cu([4]), scale=0.0)
    with pytest.raises(P.PTQError, match="UNSUPPORTED"):
        P.attn_prefill(q[..., :96].contiguous(), k[..., :96].contiguous(), k[..., :96].contiguous(), _cu([4]),
                       _cu([4]))
    with pytest.raises(P.PTQError, match="ALIGN"):
        flat = torch.zeros(4 * 2 * 128 + 8, device="cuda", dtype=torch.bfloat16)
        P.attn_prefill(q, flat[4:-4].view(4, 2, 128), k, _cu([4]), _cu([4]))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinite_keys(P, D):
    """A key whose score is -infinity counts for nothing, and a row of such keys
    alone is empty; +infinity and infinite values leave no finite row."""
    import torch

    rng = np.random.default_rng(53)
    n, nq, Hq = 200, 3, 2
    q = _values(rng, (4 * nq, Hq, D))
    k, v = (_values(rng, (4, n, 1, D)) for _ in range(2))
    q[:, :, 3] = 1.0
    k[0, 17, 0, 3] = k[1, :, 0, 3] = -np.inf
    k[2, 17, 0, 3] = np.inf
    v[3, 17, 0, 5] = np.inf
    lse = torch.full((4 * nq, Hq), 7.0, device="cuda")
    out = _host(P.attn_prefill(_dev(q), _dev(k.reshape(-1, 1, D)), _dev(v.reshape(-1, 1, D)), _cu([nq] * 4),
                               _cu([n] * 4), causal=False, lse=lse)).reshape(4, nq, Hq, D)
    lse, q = _host(lse).reshape(4, nq, Hq), q.reshape(4, nq, Hq, D)
    use = np.arange(n) != 17
    for h in range(Hq):
        ref = R.attend(q[0, :, h], k[0][use, 0], v[0][use, 0], D ** -0.5)
        R.check(out[0, :, h], lse[0, :, h], ref, True, True)
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all()
    assert np.isnan(out[2]).all() and np.isnan(lse[2]).all()
    assert (out[3, ..., 5] == np.inf).all() and np.isfinite(out[3][..., np.arange(D) != 5]).all()
