"""The attention layer's own check, on the CPU: it takes outputs that follow the formulas and refuses others."""
import math

import pytest

torch = pytest.importorskip("torch")
from bit_integer_gemm_amd import decoder  # noqa: E402


def quantise(x):
    """Levels (packed) and numbers of vectors, as the cache holds them."""
    f = x.float()
    low, high = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    scale = ((high - low) / 15).to(x.dtype)
    u = ((f - low) / scale.float()).round().clamp(0, 15).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4), torch.cat([scale, low.to(x.dtype)], -1)


def layer_by_formula(layer, cache, b, n, x, dtype):
    """(qkv, mixed, out) of sequence b's newest tokens x, the cache filled, from the definitions."""
    T, H, G, D = len(x), layer.heads, layer.kv_heads, layer.D

    def project(x, w, sw, bias):
        x = x.double()
        amax = x.abs().max(1).values[:, None]
        return ((127 * x / amax).round() @ w.double().T * amax / 127 * sw.double() + bias).to(dtype)

    qkv = project(x, layer.qkv, layer.qkv_s, layer.bias.double())
    q, k, v = qkv.view(T, H + 2 * G, D).split((H, G, G), 1)
    slots = cache.slots(torch.full((T,), b), torch.arange(n - T, n))
    for t, new in zip((0, 1), (k, v)):
        levels, numbers = quantise(new)
        cache.tensors[t][slots // cache.page, :, slots % cache.page] = levels
        cache.tensors[2 + t][slots // cache.page, :, slots % cache.page] = numbers
    mixed = torch.empty(T, H, D, dtype=dtype)
    slots = cache.slots(torch.full((n,), b), torch.arange(n))
    for h in range(H):
        vals = []
        for t in (0, 1):
            byte = cache.tensors[t][slots // cache.page, h * G // H, slots % cache.page].int()
            num = cache.tensors[2 + t][slots // cache.page, h * G // H, slots % cache.page].double()
            u = torch.empty(n, D, dtype=torch.float64)
            u[:, 0::2], u[:, 1::2] = byte % 16, byte // 16
            vals.append(u * num[:, :1] + num[:, 1:])
        for i in range(T):
            seen = n - T + i + 1
            p = torch.softmax(vals[0][:seen] @ q[i, h].double() / math.sqrt(D), 0)
            mixed[i, h] = (p @ vals[1][:seen]).to(dtype)
    return qkv, mixed, project(mixed.view(T, H * D), layer.o, layer.o_s, 0.0)


CASES = [(256, 4, 2, 64, 71, 71), (256, 4, 2, 64, 71, 1), (128, 8, 1, 128, 66, 1), (128, 2, 2, 256, 41, 41), (512, 8, 2, 128, 600, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hidden,heads,kv_heads,D,n,T", CASES)
def test_check(hidden, heads, kv_heads, D, n, T, dtype):
    g = torch.Generator().manual_seed(n + T)
    layer = decoder.Attention(hidden, heads, kv_heads, D, dtype, "cpu")
    cache = decoder.Pages(2, n, kv_heads, D, page=16, dtype=dtype, device="cpu")
    if T < n:
        layer_by_formula(layer, cache, 1, n - T, torch.randn(n - T, hidden, generator=g).to(dtype), dtype)
    x = torch.randn(T, hidden, generator=g).to(dtype)
    qkv, mixed, out = layer_by_formula(layer, cache, 1, n, x, dtype)
    decoder.check(layer, cache, 1, n, x, qkv, mixed, out)

    def refused(what, *args):
        with pytest.raises(AssertionError, match=what):
            decoder.check(layer, cache, 1, n, x, *args)

    zero = torch.zeros_like
    refused("projection", zero(qkv), mixed, out)
    refused("output projection", qkv, mixed, zero(out))
    refused("output projection", qkv, mixed, out.roll(1, 1))
    # attention that saw nothing, other heads' values, or not the last key; with the projection of that
    def project(m):
        return decoder.linear(m.reshape(T, heads * D), layer.o, layer.o_s).to(dtype)
    for wrong in (zero(mixed), mixed.roll(1, 1) if heads > 1 else -mixed, (mixed.float() * 1.05).to(dtype)):
        refused("attention", qkv, wrong, project(wrong))
    # a cache that holds another token's values in a page
    page = int(cache.table[1, 0])
    cache.tensors[1][page] = cache.tensors[1][page].roll(1, 1)
    refused("attention|cache", qkv, mixed, out)
