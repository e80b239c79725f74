"""Performance cases of the operators between a layer's projections and its
attention, and of attention over part of a paged cache:

  rope    norms of queries and keys for each head, with the position rotation
          in the same pass, positions of one or several axes (qk_rope)
  append  the same on the way into a paged key-value cache (kv_append)
  chunk   attention of each sequence's chunk of new tokens over its pages, all
          of them or a sliding window and a few first tokens (attn_chunk)
  window  the same window for one new token of each sequence (attn_decode)

`run` computes a case either with the framework's kernels (`own` true) or in
its plain form: elementary torch operations in fp32, angles in 64 bits, rounded
once at the end.  `exact` has the same outputs from the definition in 64 bits.

Layouts: a cache is pages x kv_heads x page x dim, bf16 or int8 codes, the
latter with one fp32 scale for each (page, head, token); q is (tokens, q
heads, dim), k and v (tokens, kv heads, dim); query head h reads kv head
h // group.  The widest layers here are the framework's own (hidden 5120 = 40
heads of 128); the others are generic.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BASE = 1e6

# Layers of attention heads: (kv heads, query heads per kv head, head width).
HEADS = ((8, 5, 128), (8, 4, 128), (8, 8, 128), (4, 6, 256), (2, 16, 128), (16, 1, 64), (4, 7, 64),
         (2, 10, 256), (6, 2, 128))


def listed():
    return [
        # one decode step's queries and keys for a batch of 64, normed and rotated: latency
        dict(name="rope_step", op="rope", tokens=64, kv_heads=8, group=5, dim=128, rotary=128, axes=1, pairs="half",
             norm=True, act="bf16", far=20000),
        # a long prompt of images and text: positions of time, height and width in turn
        dict(name="rope_images", op="rope", tokens=8192, kv_heads=8, group=5, dim=128, rotary=128, axes=3,
             pairs="half", norm=True, act="bf16", far=300000),
        # wide heads of which a quarter is rotated, neighbouring values in pairs, no norm, fp32, an odd number
        dict(name="rope_wide_f32", op="rope", tokens=5003, kv_heads=4, group=6, dim=256, rotary=64, axes=1,
             pairs="near", norm=False, act="f32", far=1000000),
        # the framework's fp32 decode batch (up to 8 tokens) going into an 8-bit cache: latency
        dict(name="append_step_f32_i8", op="append", tokens=8, kv_heads=8, group=5, dim=128, rotary=128, axes=1,
             pairs="half", norm=True, act="f32", kv="i8", page=64, far=30000),
        # a packed batch of prompts going into a 16-bit cache
        dict(name="append_prompt_bf16", op="append", tokens=8192, kv_heads=8, group=5, dim=128, rotary=128, axes=1,
             pairs="half", norm=True, act="bf16", kv="bf16", page=16, far=8192),
        # a long prompt of wide, partly rotated heads into an 8-bit cache, an odd number of tokens
        dict(name="append_long_i8", op="append", tokens=20011, kv_heads=4, group=6, dim=256, rotary=64, axes=1,
             pairs="half", norm=True, act="bf16", kv="i8", page=64, far=262144),
        # the few tokens that a draft of one answer is checked with, early in it: latency
        dict(name="chunk_few", op="chunk", seqs=1, min_q=4, max_q=4, prefix=777, window=0, sinks=0, kv_heads=8,
             group=5, dim=128, page=24, kv="bf16", mix=1),
        # the drafts of a serving batch checked at once, ragged lengths, 8-bit cache
        dict(name="chunk_drafts_i8", op="chunk", seqs=64, min_q=1, max_q=5, prefix=8192, window=0, sinks=0,
             kv_heads=8, group=8, dim=128, page=64, kv="i8", mix=2),
        # the next chunks of three long prompts, 16-bit cache
        dict(name="chunk_prompts", op="chunk", seqs=3, min_q=1300, max_q=2048, prefix=14000, window=0, sinks=0,
             kv_heads=8, group=5, dim=128, page=16, kv="bf16", mix=3),
        # chunks far into long texts that see a window and the first tokens, beside others' new tokens
        dict(name="chunk_window_i8", op="chunk", seqs=12, min_q=1, max_q=900, prefix=30000, window=1024, sinks=4,
             kv_heads=4, group=6, dim=256, page=64, kv="i8", mix=4),
        # a single user's token in a long answer under a window, fp32 activations: latency
        dict(name="window_one_f32", op="window", batch=1, min_len=9001, max_len=9001, window=1024, sinks=4,
             kv_heads=8, group=5, dim=128, page=16, act="f32", kv="bf16", mix=5),
        # a serving batch whose window is long, ragged lengths, 8-bit cache
        dict(name="window_64_i8", op="window", batch=64, min_len=1, max_len=30000, window=4096, sinks=16,
             kv_heads=8, group=8, dim=128, page=64, act="bf16", kv="i8", mix=6),
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    largest = {"rope": 1, "append": 5, "chunk": 8, "window": 11}
    while True:
        op = rng.choice(("rope", "append", "chunk", "chunk", "window"))
        kv_heads, group, dim = rng.choice(HEADS)
        c = dict(op=op, kv_heads=kv_heads, group=group, dim=dim)
        if op in ("rope", "append"):
            c.update(tokens=_log_int(rng, 1, 20011), rotary=rng.choice((dim, dim, dim // 2, dim // 4)),
                     axes=rng.choice((1, 1, 2, 3)), pairs=rng.choice(("half", "half", "near")),
                     norm=rng.random() < 0.7, act=rng.choice(("bf16", "f32")), far=_log_int(rng, 100, 1000000))
        if op != "rope":
            c.update(page=rng.choice((8, 16, 24, 64, 100, 256)), kv=rng.choice(("bf16", "i8")))
        if op in ("chunk", "window"):
            c.update(window=rng.choice((0, 0, 1, 1)) and _log_int(rng, 16, 8192), sinks=rng.choice((0, 1, 4, 130)),
                     mix=rng.randrange(1 << 30))
        if op == "window":
            top = _log_int(rng, 1, 65536)
            c.update(batch=_log_int(rng, 1, 128), min_len=rng.choice((0, 1, top // 2, top)), max_len=top,
                     act=rng.choice(("bf16", "f32")), window=c["window"] or 1000)
            if c["batch"] * top * kv_heads * dim > 64 * 30000 * 1024:
                continue
        elif op == "chunk":
            top = _log_int(rng, 1, 4096)
            c.update(seqs=_log_int(rng, 1, 64), min_q=rng.choice((0, 1, top)), max_q=top,
                     prefix=rng.choice((0, -(top // 2), _log_int(rng, 1, 30000), _log_int(rng, 1, 30000))))
            shown = top + (min(c["prefix"], c["window"] + c["sinks"]) if c["window"] else max(0, c["prefix"]))
            if c["seqs"] * top * kv_heads * group * shown > 40 * 3 * 2048 * 16048 or \
                    c["seqs"] * (top + max(0, c["prefix"])) * kv_heads * dim > 64 * 8192 * 1024 or \
                    sum(n for n, _ in _spans(c)) == 0:
                continue
        most, w = work(listed()[largest[op]]), work(c)
        if w["bytes"] <= max(most["bytes"], 6e8 if op == "chunk" else 0) and w["flops"] <= most["flops"] and w["bytes"] > 0:
            return c


def _lens(case):
    """The cached tokens of each sequence of a window case."""
    r = random.Random(case["mix"])
    return [r.randint(case["min_len"], case["max_len"]) for _ in range(case["batch"])]


def _spans(case):
    """(new tokens, cached tokens, the new ones among them) of each sequence of a chunk case.  A negative prefix:
    fewer tokens than queries, so that the first queries see none."""
    r = random.Random(case["mix"])
    q = [r.randint(case["min_q"], case["max_q"]) for _ in range(case["seqs"])]
    p = [r.randint(min(0, case["prefix"]), max(0, case["prefix"])) for _ in q]
    if case["seqs"] == 1:
        p = [case["prefix"]]
    return [(n, max(0, n + d)) for n, d in zip(q, p)]


def _dtype(act):
    return torch.float32 if act == "f32" else torch.bfloat16


def _new_cache(case, pages, gen):
    """A cache whose pages are full: rows of keys and values in int8 codes with their scales, whose size differs
    from row to row, or in bf16."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    if case["kv"] == "bf16":
        k, v = (torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        return dict(k=k, v=v, k_scale=None, v_scale=None)
    k, v = (torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand(shape[:3], generator=gen, device="cuda") * 0.02 + 0.008 for _ in range(2))
    return dict(k=k, v=v, k_scale=ks, v_scale=vs)


def _positions(case, gen):
    """int32, axes x tokens: running positions from some place on; further axes go through an image's rows and
    columns."""
    T = case["tokens"]
    start = int(torch.randint(0, max(1, case["far"] - T), (1,), generator=gen, device="cuda"))
    i = torch.arange(T, device="cuda")
    axis = [start + (i if case["axes"] == 1 else i // 400), (i // 20) % 20, i % 20]
    return torch.stack(axis[:case["axes"]]).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    H, G, D = case["kv_heads"], case["group"], case["dim"]
    act = _dtype(case.get("act", "bf16"))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(act)

    if case["op"] in ("rope", "append"):
        T, half = case["tokens"], case["rotary"] // 2
        # queries, keys and values as a projection gives them: side by side in one row for each token
        s["q"], s["k"], s["v"] = normal(T, H * G + 2 * H, D).split((H * G, H, H), 1)
        s["pos"] = _positions(case, gen)
        s["inv_freq"] = (BASE ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        s["axis"] = None if case["axes"] == 1 else (torch.arange(half, device="cuda") % case["axes"]).to(torch.int8)
        s["q_gain"], s["k_gain"] = (1 + 0.1 * torch.randn(D, generator=gen, device="cuda") if case["norm"] else None
                                    for _ in range(2))
        s["q_out"] = torch.empty(T, H * G, D, dtype=act, device="cuda")
        if case["op"] == "rope":
            s["k_out"] = torch.empty(T, H, D, dtype=act, device="cuda")
        else:
            pages = -(-T // case["page"]) + 3
            s["cache"] = _new_cache(case, pages, gen)
            s["slots"] = torch.randperm(pages * case["page"], generator=gen, device="cuda")[:T].to(torch.int32)
    else:
        lens = _lens(case) if case["op"] == "window" else [n for _, n in _spans(case)]
        page, wide = case["page"], max(1, -(-max(lens) // case["page"]))
        used = [-(-n // page) for n in lens]
        s["cache"] = _new_cache(case, sum(used) + 1, gen)
        order = torch.randperm(sum(used) + 1, generator=gen, device="cuda").to(torch.int32)
        col = torch.arange(wide, device="cuda")
        used = torch.tensor(used, device="cuda")
        at = (torch.cumsum(used, 0) - used)[:, None] + col
        s["table"] = torch.where(col < used[:, None], order[at.clamp(max=order.numel() - 1)], -1).to(torch.int32)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if case["op"] == "window":
            s["q"] = normal(len(lens), H * G, D)
        else:
            cu = [sum(n for n, _ in _spans(case)[:b]) for b in range(case["seqs"] + 1)]
            s["cu_q"], s["most"] = torch.tensor(cu, dtype=torch.int32, device="cuda"), max(n for n, _ in _spans(case))
            s["q"] = normal(cu[-1], H * G, D)
        s["seen"] = max(_keys(case))     # keys of the widest sequence
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device="cuda")
    if own:  # the handles and the workspace that a program keeps; nothing is computed here
        import ternary_weight_ptq1_gb300 as P

        s["P"] = P
        if "cache" in s:
            c = s["cache"]
            s["handle"] = P.KVCache(c["k"], c["v"], c["k_scale"], c["v_scale"])
        if case["op"] in ("rope", "append"):
            s["rope"] = P.Rope(s["inv_freq"], axis=s["axis"], interleaved=case["pairs"] == "near",
                               q_gain=s["q_gain"], k_gain=s["k_gain"], eps=EPS)
            if case.get("kv") == "i8":
                s["k_read"], s["v_read"] = (torch.empty(case["tokens"], H, D, dtype=torch.bfloat16, device="cuda")
                                            for _ in range(2))
        else:
            dt = P.PTQ_F32 if act == torch.float32 else P.PTQ_BF16
            if case["op"] == "window":
                need = P.attn_decode_workspace_bytes(case["batch"], H * G, H, D, dt)
            else:
                need = P.attn_chunk_workspace_bytes(case["seqs"], s["q"].shape[0], H * G, H, D, dt)
            s["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    return s


def _keys(case):
    """Cached tokens of each sequence that some query of it sees."""
    if case["op"] == "window":
        spans = [(1, n) for n in _lens(case)]
    else:
        spans = _spans(case)
    w, got = case["window"], []
    for nq, n in spans:
        lo = max(0, n - nq + 1 - w) if w else 0
        got.append(0 if nq == 0 else n - lo + min(case["sinks"], lo))
    return got


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "append": _plain_append, "chunk": _plain_attention,
            "window": _plain_attention}[state["case"]["op"]](state)


def _run_own(s):
    P, case = s["P"], s["case"]
    if case["op"] == "rope":
        q, k = P.qk_rope(s["rope"], s["q"], s["k"], s["pos"], q_out=s["q_out"], k_out=s["k_out"])
        return dict(q=q, k=k)
    if case["op"] == "append":
        q = P.kv_append(s["handle"], s["rope"], s["k"], s["v"], s["slots"], s["pos"], q=s["q"], q_out=s["q_out"])
        if case["kv"] == "bf16":
            return dict(q=q, k=s["cache"]["k"], v=s["cache"]["v"])
        k, v = P.kv_read(s["handle"], s["slots"], k=s["k_read"], v=s["v_read"])  # the values that the codes stand for
        return dict(q=q, k=k, v=v)
    if case["op"] == "window":
        out = P.attn_decode(s["q"], s["handle"], s["table"], s["lens"], window=case["window"], sinks=case["sinks"],
                            out=s["out"], lse=s["lse"], workspace=s["workspace"])
    else:
        out = P.attn_chunk(s["q"], s["handle"], s["table"], s["lens"], s["cu_q"], window=case["window"],
                           sinks=case["sinks"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return dict(out=out, lse=s["lse"])


# ---- the plain form: elementary torch operations in fp32 --------------------------------------------------------

def _plain_turned(s):
    """Queries and keys normed and rotated, in fp32."""
    case, pos = s["case"], s["pos"].double()
    R, half = case["rotary"], case["rotary"] // 2
    of_pair = pos[0][:, None] if s["axis"] is None else pos[s["axis"].long()].T        # tokens x pairs
    angle = of_pair * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x, gain):
        x = x.float()
        if gain is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain
        a, b = (x[..., :half], x[..., half:R]) if case["pairs"] == "half" else (x[..., 0:R:2], x[..., 1:R:2])
        new = (a * cos - b * sin, b * cos + a * sin)
        new = torch.cat(new, -1) if case["pairs"] == "half" else torch.stack(new, -1).flatten(-2)
        return torch.cat((new, x[..., R:]), -1)

    return turned(s["q"], s["q_gain"]), turned(s["k"], s["k_gain"])


def _plain_rope(s):
    q, k = _plain_turned(s)
    return dict(q=q.to(s["q"].dtype), k=k.to(s["k"].dtype))


def _plain_append(s):
    c, page = s["cache"], s["case"]["page"]
    q, k = _plain_turned(s)
    slots = s["slots"].long()
    page_of, at = slots // page, slots % page

    def through(x, store, scale):
        if scale is None:
            store[page_of, :, at] = x.to(torch.bfloat16)
            return store
        most = x.abs().amax(-1)
        sc = most / torch.full_like(most, 127.0)   # two tensors: a division, rounded as such
        code = torch.where(sc[..., None] > 0, torch.round(x / sc[..., None]), torch.zeros_like(x))
        store[page_of, :, at] = code.to(torch.int8)
        scale[page_of, :, at] = sc
        return (store[page_of, :, at].float() * scale[page_of, :, at][..., None]).to(torch.bfloat16)

    return dict(q=q.to(s["q"].dtype), k=through(k, c["k"], c["k_scale"]), v=through(s["v"].float(), c["v"], c["v_scale"]))


def _plain_attention(s):
    """Every sequence's queries padded to the most, its visible tokens gathered and padded likewise."""
    case, c, page = s["case"], s["cache"], s["case"]["page"]
    H, D, lens = case["kv_heads"], case["dim"], s["lens"].long()
    B = lens.numel()
    cu = torch.arange(B + 1, device=lens.device) if case["op"] == "window" else s["cu_q"].long()
    nq = cu[1:] - cu[:-1]
    most = 1 if case["op"] == "window" else s["most"]
    i = torch.arange(most, device=lens.device)
    at = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[at].transpose(1, 2).reshape(B, H, -1, most, D)                  # B, H, group, queries, D
    # the tokens that some query sees: the first ones, then those from the first query's window on
    first = (lens - nq + 1 - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(lens)
    sinks = first.clamp(max=case["sinks"])
    j = torch.arange(max(1, s["seen"]), device=lens.device)
    token = torch.where(j < sinks[:, None], j, j + (first - sinks)[:, None])            # B, keys
    there = token < lens[:, None]
    page_of = s["table"].long().gather(1, (token // page).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)

    def rows(x, scale):
        x = x[page_of, :, token % page].float()                                          # B, keys, H, D
        x = x if scale is None else x * scale[page_of, :, token % page][..., None]
        return torch.where(there[..., None, None], x, torch.zeros_like(x)).transpose(1, 2)[:, :, None]

    k, v = rows(c["k"], c["k_scale"]), rows(c["v"], c["v_scale"])
    p = (lens - nq)[:, None] + i                                                         # positions of the queries
    seen = (token[:, None] <= p[..., None]) & there[:, None] & (i < nq[:, None])[..., None]
    if case["window"]:
        seen = seen & ((token[:, None] > p[..., None] - case["window"]) | (token[:, None] < case["sinks"]))
    x = (q @ k.transpose(-1, -2)) * D ** -0.5
    x = torch.where(seen[:, None, None], x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True)
    some = torch.isfinite(top)
    w = torch.exp(x - torch.where(some, top, torch.zeros_like(top)))
    total = w.sum(-1, keepdim=True)
    out = (w @ v) / torch.where(some, total, torch.ones_like(total))
    lse = (top + torch.log(total)).squeeze(-1)
    row = (i < nq[:, None]).reshape(-1)
    out = out.reshape(B, -1, most, D).transpose(1, 2).reshape(B * most, -1, D)[row]
    lse = lse.reshape(B, -1, most).transpose(1, 2).reshape(B * most, -1)[row]
    return dict(out=out.to(s["q"].dtype), lse=lse)


# ---- the definition in 64 bits ----------------------------------------------------------------------------------

def _exact_turned(s, x, gain):
    case, x = s["case"], x.double()
    if gain is not None:
        x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * gain.double()
    R = case["rotary"]
    for n in range(R // 2):
        a, b = (n, n + R // 2) if case["pairs"] == "half" else (2 * n, 2 * n + 1)
        turn = s["pos"][n % case["axes"] if s["axis"] is not None else 0].double() * s["inv_freq"][n].double()
        z = torch.complex(x[..., a].clone(), x[..., b].clone()) * torch.polar(torch.ones_like(turn), turn)[:, None]
        x[..., a], x[..., b] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    H, G, D = case["kv_heads"], case["group"], case["dim"]
    if case["op"] in ("rope", "append"):
        q, k = _exact_turned(s, s["q"], s["q_gain"]), _exact_turned(s, s["k"], s["k_gain"])
        if case["op"] == "rope":
            return dict(q=q, k=k)
        v = s["v"].double()
        if case["kv"] == "i8":
            def step(x):
                unit = x.abs().amax(-1, keepdim=True) / 127
                return torch.where(unit > 0, (x / unit).round(), 0.0) * unit
            return dict(q=q, k=step(k), v=step(v))
        new = [s["cache"][n].double() for n in "kv"]
        where = s["slots"].long()
        for store, x in zip(new, (k, v)):
            store[where // case["page"], :, where % case["page"]] = x
        return dict(q=q, k=new[0], v=new[1])
    q = s["q"].double()
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    spans = [(1, n) for n in _lens(case)] if case["op"] == "window" else _spans(case)
    a = 0
    for b, (nq, n) in enumerate(spans):
        for h in range(H if nq and n else 0):
            pages = s["table"][b, :-(-n // case["page"])].long()
            use = torch.arange(n, device=q.device)
            if case["window"]:
                use = use[(use < case["sinks"]) | (use > n - nq - case["window"])]
            k, v = (s["cache"][x][pages[use // case["page"]], h, use % case["page"]].double() for x in "kv")
            if case["kv"] == "i8":
                k, v = (x * s["cache"][z][pages[use // case["page"]], h, use % case["page"], None]
                        for x, z in ((k, "k_scale"), (v, "v_scale")))
            rows = slice(h * G, h * G + G)
            x = torch.einsum("ihd,jd->hij", q[a:a + nq, rows], k) / math.sqrt(D)
            back = torch.arange(n - nq, n, device=q.device)[:, None] - use     # how far back a token lies
            hide = back < 0
            if case["window"]:
                hide = hide | ((back >= case["window"]) & (use >= case["sinks"]))
            x.masked_fill_(hide, -math.inf)
            total = torch.logsumexp(x, -1)
            w = torch.exp(x - total.masked_fill(total == -math.inf, 0.0)[..., None])
            out[a:a + nq, rows] = torch.einsum("hij,jd->ihd", w, v)
            lse[a:a + nq, rows] = total.T
        a += nq
    return dict(out=out, lse=lse)


# ---- what a pass cannot do without ------------------------------------------------------------------------------

def work(case):
    act = 4 if case.get("act") == "f32" else 2
    H, G, D = case["kv_heads"], case["group"], case["dim"]
    row = D * (2 if case.get("kv", "bf16") == "bf16" else 1) + (4 if case.get("kv") == "i8" else 0)
    if case["op"] in ("rope", "append"):
        T = case["tokens"]
        n = T * (H * G + H)
        flops = n * ((4 * D if case["norm"] else 0) + 3 * case["rotary"])
        if case["op"] == "rope":
            return dict(bytes=2 * n * D * act + 4 * T * case["axes"], flops=flops)
        # in: q, k and v; out: q, and the rows of the cache; in 8 bits those rows in again, and out in bf16
        back = 2 * T * H * (row + 2 * D) if case["kv"] == "i8" else 0
        return dict(bytes=T * D * act * (2 * H * G + 2 * H) + 2 * T * H * row + back + 4 * T * (1 + case["axes"]),
                    flops=flops)
    spans = [(1, n) for n in _lens(case)] if case["op"] == "window" else _spans(case)
    keys, w = _keys(case), case["window"]
    pairs = sum(min(p + 1, w + min(case["sinks"], max(0, p + 1 - w))) if w else p + 1
                for nq, n in spans for p in range(max(0, n - nq), n))
    rows = sum(nq for nq, _ in spans) * H * G
    pages = sum(-(-n // case["page"]) for n in keys)
    return dict(bytes=2 * sum(keys) * H * row + 4 * pages + rows * (2 * D * act + 4) + 8 * len(spans),
                flops=4 * pairs * H * G * D)
