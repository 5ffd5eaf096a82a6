"""The decoder layer's own check of its output projection and experts, on the CPU: it takes outputs that follow the
formulas and refuses others, at small sizes and at those that the example runs by default."""
import inspect

import pytest

torch = pytest.importorskip("torch")
from bit_integer_gemm_amd import decoder  # noqa: E402

DEFAULT = {n: inspect.signature(decoder.run_layer).parameters[n].default
           for n in ("hidden", "heads", "kv_heads", "D", "experts", "top_k", "wide", "group")}
SIZES = [dict(hidden=256, heads=4, kv_heads=2, D=64, experts=4, top_k=2, wide=128, group=64),
         dict(hidden=512, heads=8, kv_heads=1, D=128, experts=24, top_k=3, wide=96, group=32),
         {**DEFAULT, "experts": 4}]   # (an expert's sizes count, not how many there are)


@pytest.fixture(scope="module", params=range(len(SIZES)))
def layers(request):
    kept = {}
    return lambda dtype: kept.setdefault(dtype, decoder.Layer(**SIZES[request.param], dtype=dtype, device="cpu"))


def refused(what, f, *args):
    with pytest.raises(AssertionError, match=what):
        f(*args)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_output_projection(layers, dtype):
    layer = layers(dtype)
    mixed = torch.randn(5, layer.heads, layer.D, generator=torch.Generator().manual_seed(1)).mul(0.3).to(dtype)
    want = mixed.double().flatten(1) @ layer.o_value.T
    out = want.to(dtype)
    decoder.check_projection(layer, mixed, out)
    one = out.clone()
    one[3, 7] += 0.05 * want[3].square().mean().sqrt()
    for wrong in (torch.zeros_like(out), (1.05 * want).to(dtype), (want * 1.01).to(dtype), out.roll(1, 1), out.roll(1, 0), one):
        refused("output projection", decoder.check_projection, layer, mixed, wrong)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_experts(layers, dtype):
    layer = layers(dtype)
    y = torch.randn(5, layer.router.shape[1], generator=torch.Generator().manual_seed(2)).to(dtype)
    p = torch.softmax(y.double() @ layer.router.double().T, -1)
    weight, ids = p.topk(layer.top_k)

    def mix(weight, ids):
        out = torch.zeros(y.shape, dtype=torch.float64)
        for t, row in enumerate(ids.tolist()):
            for q, e in zip((weight[t] / weight[t].sum()).tolist(), row):
                gate, lift = (layer.up_value[e] @ y[t].double()).chunk(2)
                out[t] += q * (layer.down_value[e] @ (gate * torch.sigmoid(gate) * lift))
        return out

    want = mix(weight, ids)
    z = want.to(dtype)
    decoder.check_experts(layer, y, ids, z)
    one = z.clone()
    one[2, 11] += 0.05 * want[2].square().mean().sqrt()
    other = mix(weight, ids.roll(1, 1))   # the experts' weights exchanged
    for wrong in (torch.zeros_like(z), (1.05 * want).to(dtype), (1.01 * want).to(dtype), z.roll(1, 0), other.to(dtype), one):
        refused("experts", decoder.check_experts, layer, y, ids, wrong)
    least = p.topk(layer.top_k, largest=False).indices
    refused("experts", decoder.check_experts, layer, y, least, mix(p.gather(1, least), least).to(dtype))
    twice = ids[:, :1].expand(-1, layer.top_k)
    refused("experts", decoder.check_experts, layer, y, twice, mix(weight, twice).to(dtype))
