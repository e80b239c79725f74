"""One decoder layer over PTQ1_0 weights, attention and feed-forward block,
serving two requests: their prompts in chunks, then token by token.

    python examples/decoder_layer.py [--hidden 5120] [--tokens 200] [--steps 8]

The layer is pre-norm, with a norm of each query's and key's head and rotary
positions:

    x = x + Wo attention(turn(Wqkv norm(x)));   x = x + ffn(norm(x))

Every matrix is a rotated PTQ1_0 matrix (random here) applied by
rotate_matmul, the feed-forward block is ffn, and between the projections the
keys and values go through a paged int8 cache:

  prompt   bf16: kv_append norms and turns queries and keys and stores the chunk; kv_read
           returns the cached tokens, the chunk's among them, and attn_prefill sees them;
           under a window attn_chunk reads the pages.  The chunks of all requests are packed.
  decode   fp32: kv_append stores the new token, attn_decode reads the pages.

With --window W a token sees the last W tokens and the first 4.  At the end the
last token is computed again from the whole prompt (without a window by qk_rope and
attn_prefill, without a cache) and the difference is printed.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ternary_weight_ptq1_gb300 as P  # noqa: E402

D, PAGE, SINKS = 128, 64, 4


def ternary(n, k, gen):
    """A random PTQ1_0 matrix of unit gain: packed trits, scales, rotation signs."""
    trits = torch.randint(-1, 2, (n, k), generator=gen, dtype=torch.int8)
    scales = (torch.rand(n, k // 128, generator=gen) + 0.5) * (1.5 / k) ** 0.5
    signs = (torch.randint(0, 2, (k,), generator=gen) * 2 - 1).to(torch.int8)
    return (torch.from_numpy(P.pack(trits.numpy())).cuda(), scales.half().view(torch.int16).cuda(), signs.cuda())


def norm(x):
    return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)


class Layer:
    def __init__(self, hidden, q_heads, kv_heads, inner, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.hq, self.hkv = q_heads, kv_heads
        half = D // 2
        gains = [(1 + 0.1 * torch.randn(D, generator=gen)).cuda() for _ in "qk"]
        self.rope = P.Rope((1e4 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda(), q_gain=gains[0],
                           k_gain=gains[1])
        self.wqkv = ternary((q_heads + 2 * kv_heads) * D, hidden, gen)
        self.wo = ternary(hidden, q_heads * D, gen)
        self.wgu, self.wd = ternary(2 * inner, hidden, gen), ternary(hidden, inner, gen)

    def matmul(self, w, x):
        return P.rotate_matmul(w[0], w[1], x, w[2])

    def __call__(self, x, attend, act):
        """x: tokens x hidden, the fp32 residual stream; attend(q, k, v) returns
        the tokens' attention outputs; act: the projections' type, bfloat16, or
        float32 for up to 8 tokens."""
        qkv = self.matmul(self.wqkv, norm(x).to(act)).view(len(x), -1, D)
        q, k, v = qkv.split((self.hq, self.hkv, self.hkv), 1)   # columns of one row: strided
        y = attend(q, k, v)
        x = x + self.matmul(self.wo, y.reshape(len(x), -1)).float()
        y = P.ffn(self.wgu[0], self.wgu[1], self.wd[0], self.wd[1], self.wgu[2], self.wd[2], norm(x).to(act))
        return x + y.float()


class Requests:
    """The cached tokens of a batch: a page table row and a length for each."""

    def __init__(self, batch, most, layer, window=0):
        pages = -(-most // PAGE)
        self.cache = P.KVCache.empty(batch * pages, layer.hkv, PAGE, D, torch.int8)
        self.table = torch.randperm(batch * pages, device="cuda").to(torch.int32).view(batch, pages)
        self.lens = [0] * batch
        self.rope, self.window = layer.rope, dict(window=window, sinks=SINKS)

    def places(self, starts, counts):
        """Slots and positions of counts[b] tokens of each request from starts[b] on."""
        b = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).cuda()
        j = torch.cat([torch.arange(n, n + c) for n, c in zip(starts, counts)]).cuda()
        return (self.table[b, j // PAGE] * PAGE + j % PAGE).to(torch.int32), j.to(torch.int32)

    def append(self, counts, q, k, v):
        """The next counts[b] tokens of each request into the cache; their queries, normed and turned."""
        slots, pos = self.places(self.lens, counts)
        self.lens = [n + c for n, c in zip(self.lens, counts)]
        return P.kv_append(self.cache, self.rope, k, v, slots, pos, q=q)

    def prompt(self, counts):
        """attend() for the next counts[b] tokens of each request."""
        def attend(q, k, v):
            q = self.append(counts, q, k, v)
            if self.window["window"]:
                return P.attn_chunk(q, self.cache, self.table, int32(self.lens), offsets(counts), **self.window)
            # Over int8 the rows read back are the faster way for chunks of prompts (8 x 5 heads of 128: 96 tokens
            # after 96 in 11 us for attn_chunk's 22, 2048 after 2048 in 118 for 184); a few tokens each after
            # thousands are attn_chunk's (32 x 16 after 2000 in 78 for 137).
            k, v = P.kv_read(self.cache, self.places([0] * len(counts), self.lens)[0], dtype=q.dtype)
            return P.attn_prefill(q, k, v, offsets(counts), offsets(self.lens))
        return attend

    def decode(self, q, k, v):
        """attend() for one new token of every request."""
        q = self.append([1] * len(self.lens), q, k, v)
        return P.attn_decode(q, self.cache, self.table, int32(self.lens), **self.window)


def int32(values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


def offsets(lengths):
    return torch.tensor([0] + list(lengths), device="cuda").cumsum(0).to(torch.int32)


def without_cache(layer, counts):
    """attend() for whole prompts."""
    def attend(q, k, v):
        q, k = P.qk_rope(layer.rope, q, k, torch.cat([torch.arange(n) for n in counts]).to(torch.int32).cuda())
        return P.attn_prefill(q, k, v, offsets(counts), offsets(counts))
    return attend


def run(hidden=5120, q_heads=40, kv_heads=8, inner=17408, tokens=(200, 77), chunk=96, steps=8, seed=0, window=0):
    """Prompts in chunks, then decode steps; the last step's outputs, and the same
    tokens computed from the whole prompts."""
    layer = Layer(hidden, q_heads, kv_heads, inner, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = [torch.randn(n + steps, hidden, generator=gen, device="cuda") for n in tokens]
    served = Requests(len(x), max(tokens) + steps, layer, window)
    for start in range(0, max(tokens), chunk):
        counts = [max(0, min(chunk, n - start)) for n in tokens]
        rows = torch.cat([a[start:start + c] for a, c in zip(x, counts)])
        layer(rows, served.prompt(counts), torch.bfloat16)
    for i in range(steps):
        last = layer(torch.stack([a[n + i] for a, n in zip(x, tokens)]), served.decode, torch.float32)
    lens = [len(a) for a in x]
    attend = Requests(len(x), max(lens), layer, window).prompt(lens) if window else without_cache(layer, lens)
    full = layer(torch.cat(x), attend, torch.bfloat16)
    ends = torch.tensor([len(a) for a in x]).cumsum(0) - 1
    P.device_check()
    return last, full[ends.cuda()], torch.stack([a[-1] for a in x])


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--window", type=int, default=0)
    a = ap.parse_args()
    heads = a.hidden // D
    last, full, x = run(a.hidden, heads, max(1, heads // 5) if heads % 5 == 0 else max(1, heads // 4),
                        -(-17 * a.hidden // 5120) * 1024, (a.tokens, max(1, a.tokens // 3)), steps=a.steps,
                        window=a.window)
    change = (full - x).norm().item()
    print(f"the layer adds {change:.2f} to the last tokens; served token by token it differs by "
          f"{(last - full).norm().item() / change:.2e} of that")
