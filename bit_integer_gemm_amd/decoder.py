"""A decoder layer in low bits, as a server runs it.  Its attention half: int8 projections of
floating activations, a paged cache of 4-bit keys and values, attention over the cache.  The whole
layer, around the same cache and attention: norms with the residual, rotary positions, an output
projection with 4-bit weights, a mixture of experts of 4-bit weights.

    python -m bit_integer_gemm_amd.decoder

runs prompts of several lengths and then single tokens (one captured graph, replayed) through both,
with random weights, checks the outputs against the formulas in 64 bits, and prints the times.
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


def projection(name, got, want, bias):
    """One rounding of the output, and fp32 scales, product and bias before it."""
    eps, tiny = torch.finfo(got.dtype).eps, torch.finfo(got.dtype).tiny
    bound = eps / 2 * (want.abs() + tiny) + 2 ** -21 * ((want - bias).abs() + bias.abs())
    assert ((got.cpu().double() - want).abs() <= bound).all(), name


def check(layer, cache, b, n, x, qkv, mixed, out):
    """One call's projections, cache and attention of sequence b against the formulas, each from what the step before
    it left."""
    H, D, T = layer.heads, layer.D, x.shape[0]
    check_middle(layer, cache, b, n, x, qkv, qkv, mixed)
    projection("output projection", out, linear(mixed.reshape(T, H * D), layer.o, layer.o_s), torch.zeros(1).double())


def check_middle(layer, cache, b, n, x, projected, qkv, mixed):
    """The projection of x, and the cache and attention of qkv, which are its queries, keys and values, turned or not."""
    H, G, D = layer.heads, layer.kv_heads, layer.D
    T, eps, tiny = x.shape[0], torch.finfo(x.dtype).eps, torch.finfo(x.dtype).tiny
    projection("projection", projected, linear(x, layer.qkv, layer.qkv_s, layer.bias), layer.bias.cpu().double())
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


def levels4(w, group, dtype, device):
    """Weights (..., N, K) in 4 bits: packed levels, (scale, minimum) of each group of a row, and what they stand for."""
    g = w.unflatten(-1, (w.shape[-1] // group, group))
    low = g.amin(-1, keepdim=True).to(dtype)
    scale = ((g.amax(-1, keepdim=True) - low.float()) / 15).to(dtype)
    u = ((g - low.float()) / scale.float().clamp(min=1e-30)).round().clamp(0, 15)
    value = (u.double() * scale.double() + low.double()).flatten(-2)
    u = u.to(torch.uint8).flatten(-2)
    return (u[..., 0::2] | (u[..., 1::2] << 4)).to(device), torch.cat([scale, low], -1).to(device), value


class Layer:
    """r += W_o attention(rope(W_qkv norm(r))), r += post-norm of experts(norm(r)): r, the residual stream, in fp32."""

    def __init__(self, hidden, heads, kv_heads, D, experts=8, top_k=2, wide=256, group=64, dtype=torch.bfloat16,
                 device="cuda", seed=0):
        self.attention = Attention(hidden, heads, kv_heads, D, dtype, device, seed)
        self.heads, self.kv_heads, self.D, self.top_k = heads, kv_heads, D, top_k
        g = torch.Generator().manual_seed(seed + 1)

        def normal(*shape, std=1.0):
            return torch.randn(*shape, generator=g) * std

        self.o, self.o_p, self.o_value = levels4(normal(hidden, heads * D, std=(heads * D) ** -0.5), group, dtype, device)
        self.up, self.up_p, self.up_value = levels4(normal(experts, 2 * wide, hidden, std=hidden ** -0.5), group, dtype, device)
        self.down, self.down_p, self.down_value = levels4(normal(experts, hidden, wide, std=wide ** -0.5), group, dtype, device)
        self.router = normal(experts, hidden, std=2 * hidden ** -0.5).to(dtype).to(device)
        self.before, self.between, self.after = ((1 + normal(hidden, std=0.2)).to(dtype).to(device) for _ in range(3))
        self.freqs, self.mult = lb.lb_rope_freqs(D, scaling="parts", factor=4.0, before=4096.0, device=device)

    def __call__(self, r, cache, seq, pos, q_off, lens, max_q, max_len, left=None):
        """r (T, hidden) fp32, updated in place and returned; the rest as for Attention.  left: a list that receives
        what each step left, for check_layer (copies where a later step overwrites it)."""
        T, H, G, D, dtype, dev = r.shape[0], self.heads, self.kv_heads, self.D, self.before.dtype, r.device
        keep = [] if left is None else [r.clone()]
        x = torch.empty(r.shape, dtype=dtype, device=dev)
        lb.lb_residual_norm(None, r, None, x, w=self.before)
        qkv = torch.empty(T, self.attention.qkv.shape[0], dtype=dtype, device=dev)
        lb.lb_linear_w8a8(x, self.attention.qkv, self.attention.qkv_s, qkv, bias=self.attention.bias)
        if left is not None:
            keep += [x, qkv.clone()]
        q, k, v = qkv.view(T, H + 2 * G, D).split((H, G, G), 1)
        lb.lb_rope(q, k, pos, self.freqs, q, k, mult=self.mult)   # where they lie
        lb.lb_kv4_write(k, v, cache.slots(seq, pos), *cache.tensors)
        mixed = torch.empty(T, H, D, dtype=dtype, device=dev)
        lb.lb_attn_kv4(q, *cache.tensors, cache.table, q_off, lens, mixed, max_q=max_q, max_len=max_len)
        out = torch.empty_like(x)
        lb.lb_linear_w4(mixed.view(T, H * D), self.o, self.o_p, out)
        y = torch.empty_like(x)
        lb.lb_residual_norm(out, r, r, y, w=self.between)
        if left is not None:
            keep += [qkv, mixed, out, r.clone()]
        z, ids = torch.empty_like(x), torch.empty(T, self.top_k, dtype=torch.int32, device=dev)
        lb.lb_moe_w4(y, self.router, self.up, self.up_p, self.down, self.down_p, z, top_k=self.top_k, renorm=True, ids=ids)
        lb.lb_residual_norm(z, r, r, None, post_w=self.after)
        if left is not None:
            left[:] = keep + [y, ids, z, r]
        return r


EPS = 1e-5   # of the norms, lb_residual_norm's default
STEP = 2.0 ** -24


def near(name, got, want, before):
    """One rounding of the output, and `before` ahead of it."""
    eps, tiny = torch.finfo(got.dtype).eps, torch.finfo(got.dtype).tiny
    bound = eps / 2 * (want.abs() + before + tiny) + before
    assert ((got.cpu().double() - want).abs() <= bound).all(), name


def near_rows(name, got, want, before):
    """The same, and each row's error as a whole: half steps of the output bound it, with a sixteenth for what came before."""
    near(name, got, want, before)
    off = (got.cpu().double() - want).norm(dim=-1)
    assert (off <= torch.finfo(got.dtype).eps / 2 * (1 + 2 ** -4) * want.norm(dim=-1) + torch.finfo(got.dtype).tiny).all(), name


def norm(v, w):
    return v / (v.square().mean(-1, keepdim=True) + EPS).sqrt() * w.cpu().double()


def product4(x, value, numbers, off=None):
    """x W^T in 64 bits, and the square of fp32's error in it as sums of random signs have it: roundings of sums over
    16 + u in place of u and b - 16 s in place of b, two for each 16 weights and three for each group; off: the same of x."""
    scale, low = numbers.cpu().double().unbind(-1)
    size = (31 * scale.abs() + (low - 16 * scale).abs()).repeat_interleave(value.shape[-1] // scale.shape[-1], -1)
    steps = value.shape[-1] / 8 + 3 * scale.shape[-1]
    square = steps * STEP ** 2 * (x.square() @ size.square().T)
    return x @ value.T, square if off is None else square + off @ value.square().T


def check_projection(layer, mixed, out):
    want, off = product4(mixed.cpu().double().flatten(1), layer.o_value, layer.o_p)
    near_rows("output projection", out, want, 8 * off.sqrt())


def check_experts(layer, y, ids, z):
    """Experts that fp32 logits choose (two closer than their error could change places), and their products."""
    y, chosen = y.cpu().double(), ids.cpu().long()
    p = torch.softmax(y @ layer.router.cpu().double().T, -1)
    weight = p.gather(1, chosen)
    assert (weight.min(1).values >= p.topk(layer.top_k).values[:, -1] * (1 - 1e-4)).all(), "experts"
    assert all(len(set(row)) == layer.top_k for row in chosen.tolist()), "experts"
    weight = weight / weight.sum(1, keepdim=True)
    want, off = torch.zeros_like(y), torch.zeros_like(y)
    for e in chosen.unique().tolist():
        t, j = (chosen == e).nonzero(as_tuple=True)
        u, du = product4(y[t], layer.up_value[e], layer.up_p[e])
        (gate, lift), (dgate, dlift) = u.chunk(2, -1), du.chunk(2, -1)
        s = gate * torch.sigmoid(gate)
        # silu's slope is below 1.1; its own roundings and the product's: 2^-20
        dh = 1.21 * dgate * lift.square() + s.square() * dlift + (2 ** -20 * s * lift).square()
        v, dv = product4(s * lift, layer.down_value[e], layer.down_p[e], dh)
        want[t] += weight[t, j, None] * v
        # (weights: exponentials of logits off by some 2^-18)
        off[t] += weight[t, j, None] ** 2 * (dv + (2 ** -16 * v).square())
    near_rows("experts", z, want, 8 * off.sqrt())


def check_layer(layer, cache, b, n, pos, r0, x, straight, qkv, mixed, out, r1, y, ids, z, r2):
    """One call's steps for sequence b against the formulas, each from what the step before it left."""
    H, G, D = layer.heads, layer.kv_heads, layer.D
    T, att = x.shape[0], layer.attention
    r, d = r0.cpu().double(), lambda a: a.cpu().double()
    near("norm", x, norm(r, layer.before), 40 * STEP * norm(r, layer.before).abs())
    # queries and keys turned; the values as they were
    angle = d(pos)[:, None] * layer.freqs.cpu()
    c, s = (angle.cos() * layer.mult)[:, None], (angle.sin() * layer.mult)[:, None]
    before = d(straight).view(T, H + 2 * G, D)
    e, o = before[:, :H + G, :D // 2], before[:, :H + G, D // 2:]
    size = torch.cat([e.abs() + o.abs()] * 2, -1)
    after = qkv.view(T, H + 2 * G, D)
    near("rotary positions", after[:, :H + G], torch.cat([e * c - o * s, o * c + e * s], -1), 16 * STEP * layer.mult * size)
    assert torch.equal(after[:, H + G:], straight.view(T, H + 2 * G, D)[:, H + G:]), "values"
    # projection, cache and attention
    check_middle(att, cache, b, n, x, straight, qkv, mixed)
    check_projection(layer, mixed, out)
    want = r + d(out)
    near("residual", r1, want, STEP * want.abs())
    near("norm between", y, norm(want, layer.between), 40 * STEP * norm(want, layer.between).abs() + 2 * STEP)
    check_experts(layer, y, ids, z)
    want = d(r1) + norm(d(z), layer.after)
    near("residual after", r2, want, 40 * STEP * (want - d(r1)).abs() + STEP * want.abs())


def run_layer(hidden=4096, heads=32, kv_heads=8, D=128, experts=16, top_k=2, wide=1408, group=128, prompts=(100, 1, 30),
              steps=4, dtype=torch.bfloat16):
    """The whole layer: prompts, then `steps` single tokens of every sequence as a replayed graph; the times in us."""
    dev = torch.device("cuda")
    B, longest = len(prompts), max(prompts) + steps
    layer = Layer(hidden, heads, kv_heads, D, experts, top_k, wide, group, dtype, dev)
    cache = Pages(B, longest, kv_heads, D, dtype=dtype, device=dev)
    g = torch.Generator().manual_seed(3)
    start = torch.randn(sum(prompts), hidden, generator=g).to(dev)
    off = torch.tensor([0, *prompts]).cumsum(0)
    seq = torch.arange(B).repeat_interleave(torch.tensor(prompts)).to(dev)
    pos = torch.cat([torch.arange(n) for n in prompts]).to(dev)
    lens = torch.tensor(prompts, dtype=torch.int32, device=dev)
    args = (cache, seq, pos, off.to(torch.int32).to(dev), lens, max(prompts), longest)
    left = []
    layer(start.clone(), *args, left)
    for b, n in enumerate(prompts):
        check_layer(layer, cache, b, n, pos[off[b]:off[b + 1]], *(a[off[b]:off[b + 1]] for a in left))
    prefill = clock(lambda: layer(start, *args), 10)

    one = torch.empty(B, hidden, device=dev)
    every, each = torch.arange(B, device=dev), torch.arange(B + 1, dtype=torch.int32, device=dev)

    def step(left=None):
        layer(one, cache, every, lens.long() - 1, each, lens, 1, longest, left)

    one.copy_(torch.randn(B, hidden, generator=g))
    lens.add_(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # the first step, outside the graph
        step()
    torch.cuda.current_stream().wait_stream(side)
    checked, graph = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(checked):
        step(left)
    for i in range(steps):
        one.copy_(torch.randn(B, hidden, generator=g))
        if i:
            lens.add_(1)
        checked.replay()
        for b, n in enumerate(prompts):
            check_layer(layer, cache, b, n + i + 1, lens[b:b + 1] - 1, *(a[b:b + 1] for a in left))
    with torch.cuda.graph(graph):   # as it is served: without the check's copies
        step()
    one.copy_(torch.randn(B, hidden, generator=g))
    again = one.clone()
    checked.replay()
    want = one.clone()
    one.copy_(again)
    graph.replay()
    assert torch.equal(one, want), "replayed without copies"
    return prefill, clock(step, 20), clock(graph.replay, 20)


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
    for name, f in (("attention half", run), ("whole layer", run_layer)):
        prefill, eager, replayed = f()
        print(f"{name}: outputs agree; prompts {prefill:.0f} us, single tokens {eager:.0f} us, as a graph {replayed:.0f} us")
