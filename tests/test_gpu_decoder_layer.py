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
