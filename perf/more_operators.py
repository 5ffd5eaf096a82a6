"""Measured cases of the operators that complete a decoder layer in low bits.

Beside the int8 linear layer, the 4-bit cache and its attention (operators.py), such a layer needs:

  linear   out = round(sum_k x[m,k] (u[n,k] s[n,g] + b[n,g]) + bias[n]), g = k / G: weights in 4 bits, a scale and a
           minimum for each group of G of a row, on activations of 16 bits.
  moe      a whole mixture of experts for few tokens: router product, softmax, the k largest, and for each of them
           W2 (silu(Wg x) * (Wu x)) with 4-bit weights, summed with the router's weights.
  norm     what stands between two blocks: r' = r + alpha gate norm(y), x = norm(r'), norm the root-mean-square norm.
  rope     rotary positions of queries and keys: pairs in halves or side by side, part of a head, far positions.

``run`` computes them in elementary float32 torch operations, or with ``own`` set through this repository's
package; ``exact`` computes them in float64 from the definitions.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _linear(M, N, K, group, dtype, bias):
    return {"op": "linear", "M": M, "N": N, "K": K, "group": group, "dtype": dtype, "bias": bias}


def _moe(T, E, k, H, I, group, dtype, renorm):
    return {"op": "moe", "T": T, "E": E, "k": k, "H": H, "I": I, "group": group, "dtype": dtype, "renorm": renorm}


def _norm(T, H, dtype, res, post, gate, alpha):
    """gate: "" for none, "channel" for one row of numbers, "token" for a row to each token."""
    return {"op": "norm", "T": T, "H": H, "dtype": dtype, "res": res, "post": post, "gate": gate, "alpha": alpha}


def _rope(T, Hq, Hk, D, R, layout, scaling, far, dtype):
    """far: about the largest position."""
    return {"op": "rope", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "layout": layout, "scaling": scaling, "far": far,
            "dtype": dtype}


def listed():
    return [
        # One sequence generating a token: a square projection, bound by latency and by reading the weights.
        dict(_linear(1, 4096, 4096, 128, "bf16", False), name="linear4 1x4096x4096 g128"),
        # A small batch generating: the up projection, short groups, with a bias.
        dict(_linear(8, 11008, 4096, 64, "fp16", True), name="linear4 8x11008x4096 g64"),
        # Drafted tokens of a batch checked at once; rows and columns that fill no tile, the shortest groups.
        dict(_linear(61, 4097, 5504, 32, "bf16", True), name="linear4 61x4097x5504 g32"),
        # A prompt: bound by the matrix cores.
        dict(_linear(4096, 11008, 4096, 128, "bf16", False), name="linear4 4096x11008x4096 g128"),
        # One token through few, wide experts.
        dict(_moe(1, 8, 2, 4096, 11008, 128, "bf16", True), name="moe 1 token 2 of 8"),
        # A small batch through narrow experts of an odd width.
        dict(_moe(5, 64, 6, 2048, 1376, 32, "fp16", False), name="moe 5 tokens 6 of 64"),
        # A larger batch: nearly every expert is met, most by few tokens.
        dict(_moe(48, 128, 8, 2048, 1024, 128, "bf16", True), name="moe 48 tokens 8 of 128"),
        # One token between two blocks: latency.
        dict(_norm(1, 4096, "bf16", "bf16", False, "", 1.0), name="norm 1x4096"),
        # A ragged prompt with wide rows, norms on both sides of the block, a gate for each token.
        dict(_norm(777, 11008, "fp16", "fp32", True, "token", 0.7), name="norm 777x11008 token gate"),
        # A prefill batch, both norms, a gate for each channel, the residual stream in 32 bits.
        dict(_norm(8192, 4096, "bf16", "fp32", True, "channel", 1.0), name="norm 8192x4096 channel gate"),
        # Single tokens of a few sequences, far into long contexts.
        dict(_rope(5, 32, 8, 128, 128, "half", "parts", 200000, "bf16"), name="rope 5 tokens far"),
        # A prefill batch; a quarter of each head turned, pairs side by side.
        dict(_rope(8191, 32, 8, 128, 32, "pairs", "plain", 8191, "fp16"), name="rope 8191 tokens part of the head"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "moe", "norm", "rope"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "linear":
        group = rng.choice([32, 64, 128])
        M = _log(rng, 1, 64) if rng.random() < 0.7 else _log(rng, 64, 4096)
        return _linear(M, _log(rng, 512, 11008), group * _log(rng, 512 // group, 4096 // group), group, dtype, rng.random() < 0.5)
    if op == "moe":
        group = rng.choice([32, 64, 128])
        E = rng.choice([8, 16, 60, 64, 128])
        H = group * _log(rng, 1024 // group, 4096 // group)
        most = min(8192, 2 ** 28 // (E * H))  # no more weights than the listed cases have
        I = group * _log(rng, max(1, 512 // group), max(1, most // group))
        return _moe(_log(rng, 1, 64), E, rng.randrange(1, 9), H, I, group, dtype, rng.random() < 0.5)
    if op == "norm":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        H = 8 * _log(rng, 64, 2048)
        T = _log(rng, 1, 8192)
        return _norm(min(T, 2 ** 25 // H), H, dtype, rng.choice([dtype, "fp32"]), rng.random() < 0.5,
                     rng.choice(["", "channel", "token"]), rng.choice([1.0, 0.5]))
    D = rng.choice([64, 128, 256])
    Hk = rng.choice([1, 2, 4, 8])
    T = _log(rng, 1, 8192)
    Hq = min(Hk * rng.choice([1, 4, 5, 8]), max(1, 2 ** 25 // (T * D)))
    return _rope(T, Hq, Hk, D, rng.choice([D, D // 2, D // 4]), rng.choice(["half", "pairs"]),
                 rng.choice(["plain", "linear", "base", "parts", "bands"]), T + _log(rng, 10, 500000), dtype)


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    el = size[case["dtype"]]
    if case["op"] == "linear":
        M, N, K, G = case["M"], case["N"], case["K"], case["group"]
        return {"bytes": 2 * M * K + N * K // 2 + 4 * N * K // G + (2 * N if case["bias"] else 0) + 2 * M * N, "flops": 2 * M * N * K}
    if case["op"] == "moe":
        T, E, k, H, I, G = (case[n] for n in ("T", "E", "k", "H", "I", "group"))
        met = E * (1 - (1 - k / E) ** T)  # experts that some token chooses, on average
        weights = 3 * H * I
        return {"bytes": int(met * (weights // 2 + 4 * weights // G)) + 2 * E * H + 4 * T * H + 8 * T * k,
                "flops": 2 * T * (k * weights + E * H)}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        gate = {"": 0, "channel": H, "token": T * H}[case["gate"]] * el
        return {"bytes": T * H * (2 * el + 2 * size[case["res"]]) + H * el * (2 if case["post"] else 1) + gate,
                "flops": T * H * (4 + (4 if case["post"] else 0) + 3)}
    T, heads, D, R = case["T"], case["Hq"] + case["Hk"], case["D"], case["R"]
    return {"bytes": T * (2 * heads * D * el + 8) + 4 * R, "flops": T * (3 * heads * R + 10 * R)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _activations(T, H, dt, g, dev):
    """Normal activations in which a few channels are much larger than the rest."""
    x = torch.empty(T, H, device=dev).normal_(generator=g)
    x *= 1 + 20 * (torch.rand(H, generator=g, device=dev) < 0.01)
    return x.to(dt)


def _weights(lead, N, K, group, dt, g, dev):
    """Packed levels and (scale, minimum) of each group, as quantised normal weights of variance 1 / K have them."""
    lev = torch.empty(*lead, N, K, dtype=torch.float16, device=dev).normal_(7.5, 2.9, generator=g).round_().clamp_(0, 15).to(torch.uint8)
    scale = torch.empty(*lead, N, K // group, device=dev).normal_(0, 0.2, generator=g).exp_() / (2.9 * math.sqrt(K))
    low = scale * torch.empty_like(scale).normal_(-7.5, 0.4, generator=g)
    return lev[..., 0::2] | (lev[..., 1::2] << 4), torch.stack([scale, low], -1).to(dt)


def _frequencies(R, scaling):
    """Radians a position of each pair, float64, and the factor of the turned numbers, of rotary positions stretched
    eightfold beyond 4096 (the definitions: one frequency for each pair, base 10000)."""
    i = torch.arange(R // 2, dtype=torch.float64)
    f = 10000.0 ** (-2 * i / R)
    stretch, before = 8.0, 4096.0
    if scaling == "linear":
        return f / stretch, 1.0
    if scaling == "base":
        return (10000.0 * stretch ** (R / max(R - 2, 1))) ** (-2 * i / R), 1.0
    if scaling == "parts":  # whole turns within the old length: 32 and more stay, 1 and fewer are stretched
        lo, hi = (R * math.log(before / (n * 2 * math.pi)) / (2 * math.log(10000.0)) for n in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), R - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / stretch * ramp + f * (1 - ramp), 0.1 * math.log(stretch) + 1
    if scaling == "bands":  # between 1 and 4 turns within the old length, blended
        keep = ((before * f / (2 * math.pi) - 1) / 3).clamp(0, 1)
        return f / stretch * (1 - keep) + f * keep, 1.0
    return f, 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": dict(case), "op": case["op"]}
    if case["op"] == "linear":
        M, N, K, G = case["M"], case["N"], case["K"], case["group"]
        s["x"] = _activations(M, K, dt, g, dev)
        s["w"], s["p"] = _weights((), N, K, G, dt, g, dev)
        s["bias"] = torch.empty(N, device=dev).normal_(generator=g).to(dt) if case["bias"] else None
        s["out"] = torch.empty(M, N, dtype=dt, device=dev)
        return s
    if case["op"] == "moe":
        T, E, k, H, I, G = (case[n] for n in ("T", "E", "k", "H", "I", "group"))
        s["x"] = _activations(T, H, dt, g, dev)
        # logits of a spread of about two, as a trained router has them
        s["wr"] = (torch.empty(E, H, device=dev).normal_(generator=g) / math.sqrt(H)).to(dt)
        s["w1"], s["p1"] = _weights((E,), 2 * I, H, G, dt, g, dev)  # gate rows, then up rows
        s["w2"], s["p2"] = _weights((E,), H, I, G, dt, g, dev)
        s["out"] = torch.empty(T, H, dtype=dt, device=dev)
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=dev)
        s["weights"] = torch.empty(T, k, device=dev)
        return s
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        rt = DTYPES[case["res"]]
        s["y"] = _activations(T, H, dt, g, dev)
        s["r"] = (3 * torch.empty(T, H, device=dev).normal_(generator=g)).to(rt)
        s["w"] = (1 + 0.2 * torch.empty(H, device=dev).normal_(generator=g)).to(dt)
        s["wp"] = (1 + 0.2 * torch.empty(H, device=dev).normal_(generator=g)).to(dt) if case["post"] else None
        rows = {"": 0, "channel": 1, "token": T}[case["gate"]]
        gate = torch.empty(rows, H, device=dev).normal_(generator=g).to(dt) if rows else None
        s["gate"] = gate[0] if case["gate"] == "channel" else gate
        s["r_out"], s["x_out"] = torch.empty(T, H, dtype=rt, device=dev), torch.empty(T, H, dtype=dt, device=dev)
        return s
    T, Hq, Hk, D, R = (case[n] for n in ("T", "Hq", "Hk", "D", "R"))
    # queries and keys lie in the rows that the projection wrote, values behind them
    qkv = torch.empty(T, Hq + 2 * Hk, D, device=dev).normal_(generator=g).to(dt)
    s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    s["pos"] = torch.arange(T, device=dev) + (case["far"] - T if case["far"] > T else 0)
    if T < 64:  # single tokens, each of a sequence of its own
        s["pos"] = torch.randint(0, case["far"], (T,), generator=g, device=dev)
    f, s["mult"] = _frequencies(R, case["scaling"])
    s["freqs"] = f.to(dev)
    s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device=dev)
    s["k_out"] = torch.empty(T, Hk, D, dtype=dt, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_weights(packed, param):
    """The numbers that packed levels with their groups' (scale, minimum) stand for, in float32."""
    lev = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).float()
    groups = param.shape[-2]
    p = param.float()
    return (lev.unflatten(-1, (groups, -1)) * p[..., :1] + p[..., 1:]).flatten(-2)


def _plain_linear(s):
    y = s["x"].float() @ _plain_weights(s["w"], s["p"]).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    s["out"].copy_(y)
    return s["out"]


def _plain_moe(s):
    c = s["case"]
    T, E, I = c["T"], c["E"], c["I"]
    x = s["x"].float()
    p = torch.softmax(x @ s["wr"].float().t(), -1)
    # a stable sort: of equal weights the lowest index comes first
    top, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    top, ids = top[:, :c["k"]], ids[:, :c["k"]]
    if c["renorm"]:
        top = top / top.sum(-1, keepdim=True)
    share = torch.zeros(T, E, device=x.device).scatter_(1, ids, top)
    # every token through every expert, weighed by zero where it did not choose it
    u = torch.bmm(x.expand(E, -1, -1).contiguous(), _plain_weights(s["w1"], s["p1"]).transpose(1, 2).contiguous())
    h = u[..., :I] * torch.sigmoid(u[..., :I]) * u[..., I:]
    y = torch.bmm(h, _plain_weights(s["w2"], s["p2"]).transpose(1, 2).contiguous())
    s["out"].copy_((y * share.t()[..., None]).sum(0))
    s["ids"].copy_(ids)
    s["weights"].copy_(top)
    return s["out"], s["ids"], s["weights"]


EPS = 1e-5


def _plain_norm(s):
    z = s["y"].float()
    if s["wp"] is not None:
        z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * s["wp"].float()
    if s["gate"] is not None:
        z = z * s["gate"].float()
    r = s["r"].float() + s["case"]["alpha"] * z
    s["r_out"].copy_(r)
    s["x_out"].copy_(r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["w"].float())
    return s["r_out"], s["x_out"]


def _plain_turn(x, cos, sin, R, layout):
    x = x.float()
    a, b = (x[..., :R // 2], x[..., R // 2:R]) if layout == "half" else (x[..., 0:R:2], x[..., 1:R:2])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([a, b], -1) if layout == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_rope(s):
    c = s["case"]
    angle = s["pos"].double()[:, None, None] * s["freqs"]
    cos, sin = (angle.cos() * s["mult"]).float(), (angle.sin() * s["mult"]).float()
    s["q_out"].copy_(_plain_turn(s["q"], cos, sin, c["R"], c["layout"]))
    s["k_out"].copy_(_plain_turn(s["k"], cos, sin, c["R"], c["layout"]))
    return s["q_out"], s["k_out"]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    if not own:
        return {"linear": _plain_linear, "moe": _plain_moe, "norm": _plain_norm, "rope": _plain_rope}[s["op"]](s)
    import bit_integer_gemm_amd as lb
    c = s["case"]
    if s["op"] == "linear":
        if "ws" not in s:  # kept by a user's program for as long as the layer lives
            n = lb.lb_linear_w4_workspace(c["M"], c["K"], c["N"], c["group"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=s["x"].device)
        lb.lb_linear_w4(s["x"], s["w"], s["p"], s["out"], bias=s["bias"], workspace=s["ws"])
        return s["out"]
    if s["op"] == "moe":
        if "ws" not in s:
            n = lb.lb_moe_w4_workspace(c["T"], c["H"], c["I"], c["E"], c["k"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=s["x"].device)
        lb.lb_moe_w4(s["x"], s["wr"], s["w1"], s["p1"], s["w2"], s["p2"], s["out"], top_k=c["k"], renorm=c["renorm"],
                     ids=s["ids"], weights=s["weights"], workspace=s["ws"])
        return s["out"], s["ids"], s["weights"]
    if s["op"] == "norm":
        lb.lb_residual_norm(s["y"], s["r"], s["r_out"], s["x_out"], w=s["w"], post_w=s["wp"], gate=s["gate"],
                            alpha=c["alpha"], eps=EPS)
        return s["r_out"], s["x_out"]
    lb.lb_rope(s["q"], s["k"], s["pos"], s["freqs"], s["q_out"], s["k_out"], layout=c["layout"], mult=s["mult"])
    return s["q_out"], s["k_out"]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_weights(packed, param):
    """Rows of weights (N, K) in float64: level k of a row sits in nibble k % 2 of byte k / 2."""
    N, half = packed.shape
    w = torch.empty(N, 2 * half, dtype=torch.float64, device=packed.device)
    w[:, 0::2] = packed.remainder(16).double()
    w[:, 1::2] = torch.div(packed, 16, rounding_mode="floor").double()
    size = 2 * half // param.shape[1]
    scale, low = param.double().unbind(-1)
    return w.mul_(scale.repeat_interleave(size, 1)).add_(low.repeat_interleave(size, 1))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        y = torch.mm(s["x"].double(), _exact_weights(s["w"], s["p"]).t())
        return y if s["bias"] is None else y.add_(s["bias"].double()[None])
    if case["op"] == "moe":
        T, E, k, I = (case[n] for n in ("T", "E", "k", "I"))
        x = s["x"].double()
        logits = torch.mm(x, s["wr"].double().t())
        rank = [sorted(range(E), key=lambda e: (-row[e], e))[:k] for row in logits.tolist()]
        ids = torch.tensor(rank, device=x.device)
        p = logits.gather(1, ids)
        norm = torch.logsumexp(p if case["renorm"] else logits, 1, keepdim=True)
        p = torch.exp(p - norm)
        out = torch.zeros_like(x)
        for e in sorted({e for row in rank for e in row}):
            t, j = (ids == e).nonzero(as_tuple=True)
            u = torch.mm(x[t], _exact_weights(s["w1"][e], s["p1"][e]).t())
            gate, up = u[:, :I], u[:, I:]
            h = gate / (1 + torch.exp(-gate)) * up
            out[t] += p[t, j][:, None] * torch.mm(h, _exact_weights(s["w2"][e], s["p2"][e]).t())
        return out, ids.to(torch.int32), p
    if case["op"] == "norm":
        H = case["H"]
        z = s["y"].double()
        if s["wp"] is not None:
            z = z / torch.sqrt((z * z).sum(1) / H + EPS)[:, None] * s["wp"].double()
        if s["gate"] is not None:
            z = z * s["gate"].double()
        r = s["r"].double() + case["alpha"] * z
        return r, r / torch.sqrt((r * r).sum(1) / H + EPS)[:, None] * s["w"].double()
    R, got = case["R"], []
    turn = torch.polar(torch.full((1,), s["mult"], dtype=torch.float64, device=s["freqs"].device),
                       s["pos"].double()[:, None] * s["freqs"][None])[:, None]
    for x in (s["q"], s["k"]):
        y = x.double()
        if case["layout"] == "half":
            z = torch.complex(y[..., :R // 2].contiguous(), y[..., R // 2:R].contiguous()) * turn
            y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
        else:
            z = torch.complex(y[..., 0:R:2].contiguous(), y[..., 1:R:2].contiguous()) * turn
            y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
        got.append(y)
    return tuple(got)
