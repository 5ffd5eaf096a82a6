"""The attention half of a decoder layer in low bits, as a server runs it: int8 projections of
floating activations, a paged cache of 4-bit keys and values, attention over the cache.

    python -m bit_integer_gemm_amd.decoder

runs prompts of several lengths and then single tokens (one captured graph, replayed) through a
layer of random weights, checks the outputs against the formulas in 64 bits, and prints the times.
"""
import math
import time

import torch

import bit_integer_gemm_amd as lb


class Pages:
    """The cache of one layer, and the table of whose pages are whose."""

    def __init__(self, sequences, max_len, heads, D, page=64, dtype=torch.bfloat16, device="cuda"):
        self.page, width = page, -(-max_len // page)
        pages = sequences * width
        self.tensors = (torch.zeros(pages, heads, page, D // 2, dtype=torch.uint8, device=device),
                        torch.zeros(pages, heads, page, D // 2, dtype=torch.uint8, device=device),
                        torch.zeros(pages, heads, page, 2, dtype=dtype, device=device),
                        torch.zeros(pages, heads, page, 2, dtype=dtype, device=device))
        # any order will do: a server hands out pages as they become free
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32)
        self.table = order.view(sequences, width).to(device)

    def slots(self, seq, pos):
        """Slots of the tokens at positions pos of sequences seq (int64, on the GPU)."""
        return self.table[seq, pos // self.page].long() * self.page + pos % self.page


class Attention:
    """out = W_o attention(W_qkv x): W int8 with a scale for each output channel."""

    def __init__(self, hidden, heads, kv_heads, D, dtype=torch.bfloat16, device="cuda", seed=0):
        self.heads, self.kv_heads, self.D = heads, kv_heads, D
        g = torch.Generator().manual_seed(seed)
        rows = (heads + 2 * kv_heads) * D

        def weights(n, k):
            w = torch.randn(n, k, generator=g) / math.sqrt(k)
            s = w.abs().amax(1) / 127
            return (w / s[:, None]).round().to(torch.int8).to(device), s.to(device)

        self.qkv, self.qkv_s = weights(rows, hidden)
        self.bias = (torch.randn(rows, generator=g) / 8).to(dtype).to(device)
        self.o, self.o_s = weights(hidden, heads * D)

    def __call__(self, x, cache, seq, pos, q_off, lens, max_q, max_len):
        """x (T, hidden): the newest tokens of every sequence, those of one sequence next to each other;
        seq, pos (T,) int64 say which they are.  q_off, lens, max_q, max_len: as for lb_attn_kv4."""
        T, H, G, D = x.shape[0], self.heads, self.kv_heads, self.D
        qkv = torch.empty(T, self.qkv.shape[0], dtype=x.dtype, device=x.device)
        lb.lb_linear_w8a8(x, self.qkv, self.qkv_s, qkv, bias=self.bias)
        q, k, v = qkv.view(T, H + 2 * G, D).split((H, G, G), 1)   # read where they lie
        lb.lb_kv4_write(k, v, cache.slots(seq, pos), *cache.tensors)
        mixed = torch.empty(T, H, D, dtype=x.dtype, device=x.device)
        lb.lb_attn_kv4(q, *cache.tensors, cache.table, q_off, lens, mixed, max_q=max_q, max_len=max_len)
        out = torch.empty_like(x)
        lb.lb_linear_w8a8(mixed.view(T, H * D), self.o, self.o_s, out)
        return out, qkv, mixed


def linear(x, w, sw, bias=None):
    """The int8 linear layer of x (T, K) in 64 bits."""
    x = x.cpu().double()
    amax = x.abs().amax(1, keepdim=True)
    y = (127 * x / amax.clamp(min=1e-300)).round() @ w.cpu().double().T * (amax / 127) * sw.cpu().double()
    return y if bias is None else y + bias.cpu().double()


def held(cache, b, n):
    """What the cache holds for the n first tokens of sequence b, level * scale + minimum in 64 bits: keys and values
    (n, heads, D), and the largest scale of a key."""
    pos = torch.arange(n, device=cache.table.device)
    page, at = cache.table[b].long()[pos // cache.page], pos % cache.page
    found = []
    for levels, numbers in (cache.tensors[0::2], cache.tensors[1::2]):
        byte, (scale, low) = levels[page, :, at].cpu(), numbers[page, :, at].cpu().double().unbind(-1)
        u = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).double()
        found.append(u * scale[..., None] + low[..., None])
    return (*found, float(cache.tensors[2][page, :, at, 0].float().max()))


def attend(q, K, V):
    """Causal attention of the last queries q (T, H, D) over K, V (n, G, D), float64, and the largest score of
    each query and head in magnitude (T, H, 1)."""
    T, H, D = q.shape
    n, G, _ = K.shape
    K, V = (a.repeat_interleave(H // G, 1).transpose(0, 1).contiguous() for a in (K, V))
    s = torch.matmul(q.transpose(0, 1), K.transpose(1, 2)) / math.sqrt(D)
    hidden = torch.arange(n)[None, :] > torch.arange(n - T, n)[:, None]
    p = s.masked_fill(hidden, -math.inf).softmax(-1)
    return torch.matmul(p, V).transpose(0, 1), s.masked_fill(hidden, 0).abs().amax(-1).T[..., None]


def run(hidden=4096, heads=32, kv_heads=8, D=128, prompts=(777, 1, 130, 600), steps=8, dtype=torch.bfloat16):
    """Prompts, then `steps` single tokens of every sequence; returns the times in us."""
    dev = torch.device("cuda")
    B, longest = len(prompts), max(prompts) + steps
    layer = Attention(hidden, heads, kv_heads, D, dtype, dev)
    cache = Pages(B, longest, kv_heads, D, dtype=dtype, device=dev)
    g = torch.Generator().manual_seed(2)

    # the prompts, in one call
    x = torch.randn(sum(prompts), hidden, generator=g).to(dtype).to(dev)
    off = torch.tensor([0, *prompts]).cumsum(0)
    seq = torch.arange(B).repeat_interleave(torch.tensor(prompts)).to(dev)
    pos = torch.cat([torch.arange(n) for n in prompts]).to(dev)
    lens = torch.tensor(prompts, dtype=torch.int32, device=dev)
    args = (x, cache, seq, pos, off.to(torch.int32).to(dev), lens, max(prompts), longest)
    out, qkv, mixed = layer(*args)
    for b, n in enumerate(prompts):
        check(layer, cache, b, n, *(a[off[b]:off[b + 1]] for a in (x, qkv, mixed, out)))
    prefill = clock(lambda: layer(*args), 20)

    # single tokens: one graph, whose inputs and lengths move on the GPU
    one = torch.empty(B, hidden, dtype=dtype, device=dev)
    every = torch.arange(B, device=dev)
    each = torch.arange(B + 1, dtype=torch.int32, device=dev)

    def step():
        return layer(one, cache, every, lens.long() - 1, each, lens, 1, longest)

    one.copy_(torch.randn(B, hidden, generator=g))
    lens.add_(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # the first step, outside the graph
        out, qkv, mixed = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, qkv, mixed = step()
    for i in range(steps):
        if i:
            one.copy_(torch.randn(B, hidden, generator=g))
            lens.add_(1)
        graph.replay()
        for b, n in enumerate(prompts):
            check(layer, cache, b, n + i + 1, *(a[b:b + 1] for a in (one, qkv, mixed, out)))
    return prefill, clock(step, 50), clock(graph.replay, 50)


def check(layer, cache, b, n, x, qkv, mixed, out):
    """One call's projections, cache and attention of sequence b against the formulas, each from what the step before
    it left."""
    H, G, D = layer.heads, layer.kv_heads, layer.D
    T, eps, tiny = x.shape[0], torch.finfo(x.dtype).eps, torch.finfo(x.dtype).tiny
    for name, got, want, bias in (
            ("projection", qkv, linear(x, layer.qkv, layer.qkv_s, layer.bias), layer.bias.cpu().double()),
            ("output projection", out, linear(mixed.reshape(T, H * D), layer.o, layer.o_s), torch.zeros(1).double())):
        # one rounding of the output, and fp32 scales, product and bias before it
        bound = eps / 2 * (want.abs() + tiny) + 2 ** -21 * ((want - bias).abs() + bias.abs())
        assert ((got.cpu().double() - want).abs() <= bound).all(), name
    K, V, largest = held(cache, b, n)
    kv = qkv.view(T, H + 2 * G, D)[:, H:].cpu().double()
    for new, kept in ((kv[:, :G], K[n - T:]), (kv[:, G:], V[n - T:])):
        # half a level, and the scale's rounding over 15 levels
        span = new.amax(-1, keepdim=True) - new.amin(-1, keepdim=True)
        assert ((new - kept).abs() <= span / 30 + eps * span + tiny).all(), "cache"
    q = qkv.view(T, H + 2 * G, D)[:, :H].cpu().double()
    want, top = attend(q, K, V)
    # A score: D/32 products of 32 terms, about 8 rounded steps of partial sums up to 143 sum |q| each, and six more of
    # its own; the output's rounding; weights and values to 2^-10 of the weighted values' magnitudes.
    score = (D / 32 + 8) * 143 * 2 ** -23 * q.abs().sum(-1, keepdim=True) * largest / math.sqrt(D) + 6 * 2 ** -24 * (top + 1)
    mean = attend(q, K, V.abs().amax(-1, keepdim=True).expand_as(V))[0]
    bound = eps / 2 * (want.abs() + tiny) + (2 * score + 2 ** -10) * mean
    assert ((mixed.cpu().double() - want).abs() <= bound).all(), "attention"


def clock(f, n):
    """Microseconds a call, once the GPU is warm."""
    for _ in range(3):
        f()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(n):
        f()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / n * 1e6


if __name__ == "__main__":
    prefill, eager, replayed = run()
    print(f"outputs agree; prompts {prefill:.0f} us, single tokens {eager:.0f} us, as a graph {replayed:.0f} us")
