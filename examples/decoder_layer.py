"""One decoder layer over PTQ1_0 weights, attention and feed-forward block,
serving two requests: their prompts in chunks, then token by token.

    python examples/decoder_layer.py [--hidden 5120] [--tokens 200] [--steps 8]

The layer is pre-norm, without position encoding:

    x = x + Wo attention(Wqkv norm(x));   x = x + ffn(norm(x))

Every matrix is a rotated PTQ1_0 matrix (random here) applied by
rotate_matmul, the feed-forward block is ffn, and between the projections the
keys and values go through a paged int8 cache:

  prompt   bf16: kv_write stores the chunk; from the second chunk on kv_read
           returns the cached prefix and attn_prefill sees prefix and chunk
           together; the chunks of all requests are packed.
  decode   fp32: kv_write stores the new token, attn_decode reads the pages.

At the end the last token is computed again from the whole prompt and the
difference is printed.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ternary_weight_ptq1_gb300 as P  # noqa: E402

D, PAGE = 128, 64


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

    def __init__(self, batch, most, kv_heads):
        pages = -(-most // PAGE)
        self.cache = P.KVCache.empty(batch * pages, kv_heads, PAGE, D, torch.int8)
        self.table = torch.randperm(batch * pages, device="cuda").to(torch.int32).view(batch, pages)
        self.lens = [0] * batch

    def slots(self, b, start, stop):
        j = torch.arange(start, stop, device="cuda")
        return (self.table[b, j // PAGE] * PAGE + j % PAGE).to(torch.int32)

    def prompt(self, counts):
        """attend() for the next counts[b] tokens of each request."""
        def offsets(lengths):
            return torch.tensor([0] + list(lengths), device="cuda").cumsum(0).to(torch.int32)

        def attend(q, k, v):
            new = torch.cat([self.slots(b, n, n + c) for b, (n, c) in enumerate(zip(self.lens, counts))])
            P.kv_write(self.cache, k, v, new)
            ends = [n + c for n, c in zip(self.lens, counts)]
            if any(self.lens):      # the prefix as it is stored, and the chunk
                k, v = P.kv_read(self.cache, torch.cat([self.slots(b, 0, e) for b, e in enumerate(ends)]),
                                 dtype=q.dtype)
            self.lens = ends
            return P.attn_prefill(q, k, v, offsets(counts), offsets(ends))
        return attend

    def decode(self, q, k, v):
        """attend() for one new token of every request."""
        P.kv_write(self.cache, k, v, torch.cat([self.slots(b, n, n + 1) for b, n in enumerate(self.lens)]))
        self.lens = [n + 1 for n in self.lens]
        return P.attn_decode(q, self.cache, self.table, torch.tensor(self.lens, dtype=torch.int32, device="cuda"))


def run(hidden=5120, q_heads=40, kv_heads=8, inner=17408, tokens=(200, 77), chunk=96, steps=8, seed=0):
    """Prompts in chunks, then decode steps; the last step's outputs, and the same
    tokens computed from the whole prompts."""
    layer = Layer(hidden, q_heads, kv_heads, inner, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = [torch.randn(n + steps, hidden, generator=gen, device="cuda") for n in tokens]
    served = Requests(len(x), max(tokens) + steps, kv_heads)
    for start in range(0, max(tokens), chunk):
        counts = [max(0, min(chunk, n - start)) for n in tokens]
        rows = torch.cat([a[start:start + c] for a, c in zip(x, counts)])
        layer(rows, served.prompt(counts), torch.bfloat16)
    for i in range(steps):
        last = layer(torch.stack([a[n + i] for a, n in zip(x, tokens)]), served.decode, torch.float32)
    whole = Requests(len(x), max(tokens) + steps, kv_heads)
    full = layer(torch.cat(x), whole.prompt([len(a) for a in x]), torch.bfloat16)
    ends = torch.tensor([len(a) for a in x]).cumsum(0) - 1
    P.device_check()
    return last, full[ends.cuda()], torch.stack([a[-1] for a in x])


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    heads = a.hidden // D
    last, full, x = run(a.hidden, heads, max(1, heads // 5) if heads % 5 == 0 else max(1, heads // 4),
                        -(-17 * a.hidden // 5120) * 1024, (a.tokens, max(1, a.tokens // 3)), steps=a.steps)
    change = (full - x).norm().item()
    print(f"the layer adds {change:.2f} to the last tokens; served token by token it differs by "
          f"{(last - full).norm().item() / change:.2e} of that")
