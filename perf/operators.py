"""Performance cases of the attention operators: the paged key-value cache
(kv_write, kv_read), the attention of one new token over it (attn_decode) and
the attention of whole prompts (attn_prefill).

`run` computes a case either with the framework's kernels (`own` true) or in
its plain form: elementary torch operations in fp32, rounded once at the end.
`exact` has the same outputs from the definition in 64 bits.

Layouts: a cache is pages x kv_heads x page x dim, bf16 or int8 codes, the
latter with one fp32 scale for each (page, head, token); q is (tokens, q
heads, dim), k and v (tokens, kv heads, dim); query head h reads kv head
h // group.  The largest activation widths here are the framework's own
(hidden 5120 = 40 heads of 128); the others are generic.
"""
import math
import random

import torch

own = False

# Layers of attention heads: (kv heads, query heads per kv head, head width).
HEADS = ((8, 5, 128), (8, 4, 128), (8, 8, 128), (4, 6, 256), (2, 16, 128), (16, 1, 64), (4, 7, 64),
         (2, 10, 256), (1, 20, 64), (6, 2, 128))


def listed():
    return [
        # one decode step's new tokens, a token for each of 64 sequences: latency
        dict(name="cache_step_f32_i8", op="cache", tokens=64, kv_heads=8, dim=128, page=64, act="f32", kv="i8"),
        # a packed batch of prompts going into an 8-bit cache and back out as a prefix
        dict(name="cache_prompt_bf16_i8", op="cache", tokens=8192, kv_heads=8, dim=128, page=64, act="bf16", kv="i8"),
        # a long prompt of wide heads through a 16-bit cache, an odd number of tokens
        dict(name="cache_long_bf16_bf16", op="cache", tokens=33001, kv_heads=4, dim=256, page=16, act="bf16", kv="bf16"),
        # a single user's token early in an answer, fp32 activations: latency
        dict(name="decode_one_f32_bf16", op="decode", batch=1, min_len=777, max_len=777, kv_heads=8, group=5, dim=128,
             page=16, act="f32", kv="bf16", mix=1),
        # the framework's fp32 decode batch (up to 8 tokens) over an 8-bit cache, ragged
        dict(name="decode_8_f32_i8", op="decode", batch=8, min_len=1, max_len=4096, kv_heads=8, group=5, dim=128,
             page=64, act="f32", kv="i8", mix=2),
        # a serving batch, ragged lengths, 8-bit cache: the ordinary case
        dict(name="decode_64_bf16_i8", op="decode", batch=64, min_len=1, max_len=8192, kv_heads=8, group=8, dim=128,
             page=64, act="bf16", kv="i8", mix=3),
        # one very long context, wide heads, 16-bit cache
        dict(name="decode_long_bf16_bf16", op="decode", batch=1, min_len=131001, max_len=131001, kv_heads=4, group=6,
             dim=256, page=16, act="bf16", kv="bf16", mix=4),
        # many short sequences, a kv head for each query head, pages of an odd size
        dict(name="decode_96_bf16_mha", op="decode", batch=96, min_len=0, max_len=700, kv_heads=16, group=1, dim=64,
             page=24, act="bf16", kv="bf16", mix=5),
        # one short question: latency
        dict(name="prefill_short", op="prefill", seqs=1, min_q=77, max_q=77, prefix=0, kv_heads=8, group=5, dim=128,
             causal=True, mix=6),
        # a packed batch of prompts of different lengths
        dict(name="prefill_packed", op="prefill", seqs=16, min_q=1, max_q=1100, prefix=0, kv_heads=8, group=5,
             dim=128, causal=True, mix=7),
        # one long prompt
        dict(name="prefill_long", op="prefill", seqs=1, min_q=8192, max_q=8192, prefix=0, kv_heads=8, group=5,
             dim=128, causal=True, mix=8),
        # the next chunks of two prompts over the prefixes that were read back from the cache, wide heads
        dict(name="prefill_prefix_wide", op="prefill", seqs=2, min_q=401, max_q=515, prefix=7000, kv_heads=4,
             group=6, dim=256, causal=True, mix=9),
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(("cache", "decode", "decode", "prefill", "prefill"))
        kv_heads, group, dim = rng.choice(HEADS)
        page = rng.choice((8, 16, 24, 64, 100, 256))
        mix = rng.randrange(1 << 30)
        if op == "cache":
            c = dict(op=op, tokens=_log_int(rng, 1, 32768), kv_heads=kv_heads, dim=dim, page=page,
                     act=rng.choice(("bf16", "f32")), kv=rng.choice(("bf16", "i8")))
            if c["tokens"] * kv_heads * dim <= 33001 * 1024 and c["tokens"] != 3072:
                return c
        elif op == "decode":
            top = _log_int(rng, 1, 131072)
            c = dict(op=op, batch=_log_int(rng, 1, 256), min_len=rng.choice((0, 1, top // 2, top)), max_len=top,
                     kv_heads=kv_heads, group=group, dim=dim, page=page, act=rng.choice(("bf16", "f32")),
                     kv=rng.choice(("bf16", "i8")), mix=mix)
            if c["batch"] * top * kv_heads * dim <= 64 * 8192 * 1024 and top != 3072 and \
                    work(c)["bytes"] <= work(listed()[5])["bytes"]:
                return c
        else:
            top = _log_int(rng, 1, 8192)
            c = dict(op=op, seqs=_log_int(rng, 1, 24), min_q=rng.choice((0, 1, top)), max_q=top,
                     prefix=rng.choice((0, 0, -(top // 2), _log_int(rng, 1, 8192))), kv_heads=kv_heads, group=group,
                     dim=dim, causal=rng.random() < 0.75, mix=mix)
            if c["seqs"] * kv_heads * group * top * (top + max(0, c["prefix"])) <= 40 * 8192 * 8192 and \
                    3072 not in (top, c["prefix"]) and work(c)["flops"] <= work(listed()[10])["flops"] and \
                    sum(n for n, _ in _spans(c)) > 0:
                return c


def _lens(case):
    """The cached tokens of each sequence of a decode case."""
    r = random.Random(case["mix"])
    return [r.randint(case["min_len"], case["max_len"]) for _ in range(case["batch"])]


def _spans(case):
    """(queries, keys) of each sequence of a prefill case.  A negative prefix: fewer keys than queries, so that
    under the causal mask the first queries see none."""
    r = random.Random(case["mix"])
    q = [r.randint(case["min_q"], case["max_q"]) for _ in range(case["seqs"])]
    p = [r.randint(min(0, case["prefix"]), max(0, case["prefix"])) for _ in q]
    return [(n, max(0, n + d)) for n, d in zip(q, p)]


def _dtype(act):
    return torch.float32 if act == "f32" else torch.bfloat16


def _new_cache(case, tokens, gen):
    """A cache with room for `tokens` tokens, and every page in use filled: rows of keys and values whose size
    differs from token to token, in int8 codes with their scales, or rounded to bf16."""
    pages = max(1, -(-tokens // case["page"]))
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    if case["kv"] == "bf16":
        k, v = (torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        return dict(k=k, v=v, k_scale=None, v_scale=None)
    k, v = (torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand(shape[:3], generator=gen, device="cuda") * 0.02 + 0.008 for _ in range(2))
    return dict(k=k, v=v, k_scale=ks, v_scale=vs)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = dict(case=case)
    act = _dtype(case.get("act", "bf16"))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(act)

    if case["op"] == "cache":
        T, H, D = case["tokens"], case["kv_heads"], case["dim"]
        state["cache"] = _new_cache(case, T + 3 * case["page"], gen)
        room = state["cache"]["k"].shape[0] * case["page"]
        state["slots"] = torch.randperm(room, generator=gen, device="cuda")[:T].to(torch.int32)
        # keys and values as a projection gives them: side by side in one row for each token
        kv = normal(T, 2, H, D)
        state["k"], state["v"] = kv[:, 0], kv[:, 1]
    elif case["op"] == "decode":
        B, H, G, D, page = case["batch"], case["kv_heads"], case["group"], case["dim"], case["page"]
        lens = _lens(case)
        wide = max(1, -(-max(lens) // page))
        used = [-(-n // page) for n in lens]
        state["cache"] = _new_cache(case, (sum(used) + 1) * page, gen)
        order = torch.randperm(sum(used) + 1, generator=gen, device="cuda").to(torch.int32)
        col = torch.arange(wide, device="cuda")
        used = torch.tensor(used, device="cuda")
        at = (torch.cumsum(used, 0) - used)[:, None] + col
        state["table"] = torch.where(col < used[:, None], order[at.clamp(max=order.numel() - 1)], -1).to(torch.int32)
        state["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        state["q"] = normal(B, H * G, D)
        state["out"], state["lse"] = torch.empty_like(state["q"]), torch.empty(B, H * G, device="cuda")
    else:
        H, G, D = case["kv_heads"], case["group"], case["dim"]
        spans = _spans(case)
        state["cu_q"], state["cu_k"] = (
            torch.tensor([0] + [sum(s[i] for s in spans[:n + 1]) for n in range(len(spans))], dtype=torch.int32,
                         device="cuda") for i in (0, 1))
        state["most"] = tuple(max(s[i] for s in spans) for i in (0, 1))
        state["q"] = normal(sum(s[0] for s in spans), H * G, D)
        state["k"], state["v"] = (normal(sum(s[1] for s in spans), H, D) for _ in range(2))
        state["out"], state["lse"] = torch.empty_like(state["q"]), torch.empty(state["q"].shape[:2], device="cuda")
    if own:  # the handle and the workspace that a program keeps beside its cache; nothing is computed here
        import ternary_weight_ptq1_gb300 as P

        state["P"] = P
        if "cache" in state:
            c = state["cache"]
            state["handle"] = P.KVCache(c["k"], c["v"], c["k_scale"], c["v_scale"])
        dt = P.PTQ_F32 if act == torch.float32 else P.PTQ_BF16
        need = 0
        if case["op"] == "decode":
            need = P.attn_decode_workspace_bytes(case["batch"], case["kv_heads"] * case["group"], case["kv_heads"],
                                                 case["dim"], dt)
        elif case["op"] == "prefill":
            need = P.attn_prefill_workspace_bytes(case["seqs"], state["q"].shape[0], state["k"].shape[0],
                                                  case["kv_heads"] * case["group"], case["kv_heads"], case["dim"], dt)
        state["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    return state


def run(state):
    if own:
        return _run_own(state)
    return {"cache": _plain_cache, "decode": _plain_decode, "prefill": _plain_prefill}[state["case"]["op"]](state)


def _run_own(s):
    P, op = s["P"], s["case"]["op"]
    if op == "cache":
        P.kv_write(s["handle"], s["k"], s["v"], s["slots"])
        k, v = P.kv_read(s["handle"], s["slots"], dtype=s["k"].dtype)
        return dict(k=k, v=v)
    if op == "decode":
        out = P.attn_decode(s["q"], s["handle"], s["table"], s["lens"], out=s["out"], lse=s["lse"],
                            workspace=s["workspace"])
    else:
        out = P.attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=s["case"]["causal"], out=s["out"],
                             lse=s["lse"], workspace=s["workspace"])
    return dict(out=out, lse=s["lse"])


# ---- the plain form: elementary torch operations in fp32 --------------------------------------------------------

def _plain_cache(s):
    c, page = s["cache"], s["case"]["page"]
    slots = s["slots"].long()
    page_of, at = slots // page, slots % page

    def through(x, store, scale):
        x = x.float()
        if scale is None:
            store[page_of, :, at] = x.to(torch.bfloat16)
            return store[page_of, :, at].to(s["k"].dtype)
        most = x.abs().amax(-1)
        sc = most / torch.full_like(most, 127.0)   # two tensors: a division, rounded as such
        code = torch.where(sc[..., None] > 0, torch.round(x / sc[..., None]), torch.zeros_like(x))
        store[page_of, :, at] = code.to(torch.int8)
        scale[page_of, :, at] = sc
        return (store[page_of, :, at].float() * scale[page_of, :, at][..., None]).to(s["k"].dtype)

    return dict(k=through(s["k"], c["k"], c["k_scale"]), v=through(s["v"], c["v"], c["v_scale"]))


def _softmax_sum(scores, seen, v):
    """The attention's output and its log-sum-exp from scores (..., queries, keys), which of them count, and
    values (..., keys, dim); 0 and -inf where none counts."""
    scores = torch.where(seen, scores, torch.full_like(scores, -math.inf))
    top = scores.amax(-1, keepdim=True)
    some = torch.isfinite(top)
    p = torch.exp(scores - torch.where(some, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(some, total, torch.ones_like(total))
    return out, (top + torch.log(total)).squeeze(-1)


def _plain_decode(s):
    c, q, table = s["cache"], s["q"].float(), s["table"].clamp(min=0).long()
    B, H, D = q.shape[0], c["k"].shape[1], q.shape[2]
    some = torch.arange(table.shape[1] * c["k"].shape[2], device=q.device) < s["lens"][:, None]  # B x tokens

    def gathered(x, scale):
        x = x[table].float()                                    # B, pages, H, page, D
        x = x if scale is None else x * scale[table][..., None]
        x = x.transpose(1, 2).reshape(B, H, -1, D)
        return torch.where(some[:, None, :, None], x, torch.zeros_like(x))

    k, v = gathered(c["k"], c["k_scale"]), gathered(c["v"], c["v_scale"])
    scores = (q.reshape(B, H, -1, D) @ k.transpose(-1, -2)) * D ** -0.5
    out, lse = _softmax_sum(scores, some[:, None, None], v)
    return dict(out=out.reshape(s["q"].shape).to(s["q"].dtype), lse=lse.reshape(B, -1))


def _plain_prefill(s):
    """Every sequence padded to the longest."""
    (nq, nk), cu_q, cu_k = s["most"], s["cu_q"].long(), s["cu_k"].long()
    B, H, D = cu_q.numel() - 1, s["k"].shape[1], s["q"].shape[2]
    i, j = torch.arange(nq, device=cu_q.device), torch.arange(nk, device=cu_q.device)
    lq, lk = (cu_q[1:] - cu_q[:-1])[:, None], (cu_k[1:] - cu_k[:-1])[:, None]

    def padded(x, cu, at, n):
        x = x[(cu[:-1, None] + at).clamp(max=x.shape[0] - 1)].float() if x.shape[0] else \
            x.new_zeros((B, at.numel()) + x.shape[1:], dtype=torch.float32)
        return torch.where((at < n)[..., None, None], x, torch.zeros_like(x)).transpose(1, 2)  # B, heads, tokens, D

    q = padded(s["q"], cu_q, i, lq).reshape(B, H, -1, nq, D)
    k, v = padded(s["k"], cu_k, j, lk)[:, :, None], padded(s["v"], cu_k, j, lk)[:, :, None]
    seen = (i < lq)[:, :, None] & (j < lk)[:, None, :]
    if s["case"]["causal"]:
        seen = seen & (j <= (i + lk - lq)[:, :, None])
    if nk:
        out, lse = _softmax_sum((q @ k.transpose(-1, -2)) * D ** -0.5, seen[:, None, None], v)
    else:
        out, lse = torch.zeros_like(q), torch.full_like(q[..., 0], -math.inf)
    row = (i < lq).reshape(-1)
    out = out.reshape(B, -1, nq, D).transpose(1, 2).reshape(B * nq, -1, D)[row]
    lse = lse.reshape(B, -1, nq).transpose(1, 2).reshape(B * nq, -1)[row]
    return dict(out=out.to(s["q"].dtype), lse=lse)


# ---- the definition in 64 bits ----------------------------------------------------------------------------------

def _exact_row_block(q, k, v, shown):
    """q: heads x queries x dim, k and v: keys x dim, shown: queries x keys; one sequence, one kv head."""
    x = torch.einsum("gid,jd->gij", q, k) / math.sqrt(q.shape[-1])
    x = x.masked_fill(~shown, -math.inf)
    lse = torch.logsumexp(x, -1)
    w = torch.exp(x - lse.masked_fill(lse == -math.inf, 0.0)[..., None])
    return torch.einsum("gij,jd->gid", w, v), lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "cache":
        def value(x):
            x = x.double()
            if case["kv"] == "bf16":
                return x.to(torch.bfloat16).double()
            step = x.abs().amax(-1, keepdim=True) / 127
            return torch.where(step > 0, (x / step).round(), 0.0) * step
        return dict(k=value(s["k"]), v=value(s["v"]))
    H, G, D = case["kv_heads"], case["group"], case["dim"]
    q = s["q"].double()
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    if case["op"] == "decode":
        for b, n in enumerate(_lens(case)):
            if n == 0:
                continue
            pages = s["table"][b, :-(-n // case["page"])].long()
            k, v = (s["cache"][x][pages].double() for x in "kv")
            if case["kv"] == "i8":
                k, v = k * s["cache"]["k_scale"][pages][..., None], v * s["cache"]["v_scale"][pages][..., None]
            for h in range(H):
                rows = slice(h * G, h * G + G)
                o, l = _exact_row_block(q[b, rows, None], k[:, h].reshape(-1, D)[:n], v[:, h].reshape(-1, D)[:n],
                                        torch.ones(1, n, dtype=torch.bool, device=q.device))
                out[b, rows], lse[b, rows] = o[:, 0], l[:, 0]
        return dict(out=out, lse=lse)
    aq = ak = 0
    for nq, nk in _spans(case):
        i, j = torch.arange(nq, device=q.device)[:, None], torch.arange(nk, device=q.device)
        shown = (j - i <= nk - nq) if case["causal"] else (j >= 0).expand(nq, nk)
        for h in range(H if nq and nk else 0):
            rows = slice(h * G, h * G + G)
            o, l = _exact_row_block(q[aq:aq + nq, rows].transpose(0, 1), s["k"][ak:ak + nk, h].double(),
                                    s["v"][ak:ak + nk, h].double(), shown)
            out[aq:aq + nq, rows], lse[aq:aq + nq, rows] = o.transpose(0, 1), l.transpose(0, 1)
        aq, ak = aq + nq, ak + nk
    return dict(out=out, lse=lse)


# ---- what a pass cannot do without ------------------------------------------------------------------------------

def work(case):
    act = 4 if case.get("act") == "f32" else 2
    D = case["dim"]
    row = D * (2 if case.get("kv", "bf16") == "bf16" else 1) + (4 if case.get("kv") == "i8" else 0)
    if case["op"] == "cache":
        # in: k and v; out: their rows of the cache; then the rows in and k and v out
        n = 2 * case["tokens"] * case["kv_heads"]
        return dict(bytes=2 * n * (D * act + row) + 8 * case["tokens"], flops=4 * n * D)
    heads = case["kv_heads"] * case["group"]
    if case["op"] == "decode":
        lens = _lens(case)
        seen, pages = sum(lens), sum(-(-n // case["page"]) for n in lens)
        return dict(bytes=2 * seen * case["kv_heads"] * row + 4 * pages + case["batch"] * (4 + heads * (2 * D * act + 4)),
                    flops=4 * seen * heads * D)
    spans = _spans(case)
    pairs = sum(sum(max(0, min(nk, i + 1 + nk - nq)) for i in range(nq)) if case["causal"] else nq * nk
                for nq, nk in spans)
    tq, tk = sum(s[0] for s in spans), sum(s[1] for s in spans)
    return dict(bytes=tq * heads * (2 * D * act + 4) + 2 * tk * case["kv_heads"] * D * act, flops=4 * pairs * heads * D)
