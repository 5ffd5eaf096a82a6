"""The whole decoder layer: every operator in its place, prompts, then single tokens as a replayed graph."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("hidden,heads,kv_heads,D,experts,top_k,wide,group,prompts", [
    (256, 4, 2, 64, 4, 2, 128, 64, (1, 70, 33)),
    (512, 8, 1, 128, 24, 3, 96, 32, (65, 16)),
    (512, 2, 2, 256, 8, 1, 256, 128, (40,)),
])
def test_prompts_then_tokens(hidden, heads, kv_heads, D, experts, top_k, wide, group, prompts, dtype):
    from bit_integer_gemm_amd import decoder
    decoder.run_layer(hidden, heads, kv_heads, D, experts, top_k, wide, group, prompts, steps=3, dtype=getattr(torch, dtype))


def test_serving_makes_no_copies():
    """The check's copies are made for the check alone; the residual stream comes out the same."""
    from torch.overrides import TorchFunctionMode

    from bit_integer_gemm_amd import decoder

    class Clones(TorchFunctionMode):
        made = 0

        def __torch_function__(self, func, types, args=(), kwargs=None):
            self.made += getattr(func, "__name__", "") == "clone"
            return func(*args, **(kwargs or {}))

    layer = decoder.Layer(256, 4, 2, 64, experts=4, top_k=2, wide=128, group=64)
    start = torch.randn(5, 256, generator=torch.Generator().manual_seed(4)).cuda()
    off, lens = torch.tensor([0, 5], dtype=torch.int32, device="cuda"), torch.tensor([5], dtype=torch.int32, device="cuda")
    seq, pos = torch.zeros(5, dtype=torch.int64, device="cuda"), torch.arange(5, device="cuda")
    got = []
    for left in (None, []):
        r = start.clone()
        with Clones() as clones:
            same = layer(r, decoder.Pages(1, 5, 2, 64, device="cuda"), seq, pos, off, lens, 5, 5, left)
        assert same is r and clones.made == (0 if left is None else 3)
        got.append(r)
    assert torch.equal(*got) and torch.equal(left[0], start) and left[-1] is got[1]
