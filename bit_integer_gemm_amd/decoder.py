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


def reference(layer, x, cache, b, n):
    """In 64 bits: the projection of sequence b's newest tokens x, and the n keys and values that the
    cache holds for it."""
    G, D = layer.kv_heads, layer.D
    x = x.cpu().double()
    amax = x.abs().amax(1, keepdim=True)
    qkv = (127 * x / amax).round() @ layer.qkv.cpu().double().T * (amax / 127) * layer.qkv_s.cpu().double()
    qkv += layer.bias.cpu().double()
    pos = torch.arange(n, device=cache.table.device)
    K = torch.empty(n, G, D, dtype=layer.bias.dtype, device=pos.device)
    V = torch.empty_like(K)
    lb.lb_kv4_read(*cache.tensors, cache.slots(torch.full_like(pos, b), pos), K, V)
    return qkv, K.cpu().double(), V.cpu().double()


def attend(q, K, V):
    """Causal attention of the last queries q (T, H, D) over K, V (n, G, D), float64."""
    T, H, D = q.shape
    n, G, _ = K.shape
    K, V = (a.repeat_interleave(H // G, 1).transpose(0, 1).contiguous() for a in (K, V))
    s = torch.matmul(q.transpose(0, 1), K.transpose(1, 2)) / math.sqrt(D)
    hidden = torch.arange(n)[None, :] > torch.arange(n - T, n)[:, None]
    p = s.masked_fill(hidden, -math.inf).softmax(-1)
    return torch.matmul(p, V).transpose(0, 1)


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
    _, qkv, mixed = layer(*args)
    for b, n in enumerate(prompts):
        check(layer, cache, b, n, x[off[b]:off[b + 1]], qkv[off[b]:off[b + 1]], mixed[off[b]:off[b + 1]])
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
            check(layer, cache, b, n + i + 1, one[b:b + 1], qkv[b:b + 1], mixed[b:b + 1])
    return prefill, clock(step, 50), clock(graph.replay, 50)


def check(layer, cache, b, n, x, qkv, mixed):
    """One call's projection and attention of sequence b against the formulas."""
    H, G, D = layer.heads, layer.kv_heads, layer.D
    T, eps, tiny = x.shape[0], torch.finfo(x.dtype).eps, torch.finfo(x.dtype).tiny
    want, K, V = reference(layer, x, cache, b, n)
    # one rounding of the output, and fp32 scales, product and bias before it
    bias = layer.bias.cpu().double()
    bound = eps / 2 * (want.abs() + tiny) + 2 ** -21 * ((want - bias).abs() + bias.abs())
    assert ((qkv.cpu().double() - want).abs() <= bound).all(), "projection"
    kv = qkv.view(T, H + 2 * G, D)[:, H:].cpu().double()
    for new, held in ((kv[:, :G], K[n - T:]), (kv[:, G:], V[n - T:])):
        # half a level and the scale's rounding over 15 levels; one rounding each of minimum and result
        span = new.amax(-1, keepdim=True) - new.amin(-1, keepdim=True)
        assert ((new - held).abs() <= span / 30 + eps * span + eps * new.abs().amax(-1, keepdim=True)).all(), "cache"
    q = qkv.view(T, H + 2 * G, D)[:, :H].cpu().double()
    # the output's rounding, and that of what is read back (K moves the scores by |q| |K| eps/2 sqrt(D) at most)
    bound = 4 * eps * (1 + q.norm(dim=-1).amax() * K.norm(dim=-1).amax() / math.sqrt(D)) * V.abs().amax()
    assert ((mixed.cpu().double() - attend(q, K, V)).abs() <= bound).all(), "attention"


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
