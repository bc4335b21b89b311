"""The example runs the MX4 products and the block-quantized cache together and checks each step itself."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mx4_attention_layer.py")


@pytest.mark.parametrize("type_,heads,kv_heads,d,prompts,drafts", [("q8_0", 8, 2, 64, (100, 37), (6, 4)), ("q4_0", 8, 8, 128, (65, 1), (1, 3)),
                                                                   ("q8_0", 16, 1, 96, (200, 130), (17, 8))])
def test_example(type_, heads, kv_heads, d, prompts, drafts):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gb300 import build

    build.build()
    spec = importlib.util.spec_from_file_location("mx4_attention_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(type_, heads=heads, kv_heads=kv_heads, d=d, prompts=prompts, drafts=drafts) == [a + b for a, b in zip(prompts, drafts)]
