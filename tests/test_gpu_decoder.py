"""The attention layer that runs the serving operators together: prompts, then single tokens."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("hidden,heads,kv_heads,D,prompts", [
    (256, 4, 2, 64, (1, 70, 33)),
    (512, 8, 1, 128, (65, 16)),
    (512, 2, 2, 256, (40,)),
])
def test_prompts_then_tokens(hidden, heads, kv_heads, D, prompts, dtype):
    from bit_integer_gemm_amd import decoder
    decoder.run(hidden, heads, kv_heads, D, prompts, steps=4, dtype=getattr(torch, dtype))
