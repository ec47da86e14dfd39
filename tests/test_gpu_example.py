"""The example that uses the 8-bit operators together, at small odd sizes."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens,channels,hidden,experts,top,vocab", [
    (1, 512, 256, 8, 2, 1000), (77, 528, 272, 5, 1, 520), (300, 1024, 512, 16, 3, 2048)])
def test_fp8_block_is_near_the_plain_block(tokens, channels, hidden, experts, top, vocab):
    import tma_pipelined_tensor_tn_gb300 as tg
    tg.build()
    spec = importlib.util.spec_from_file_location(
        "fp8_moe_block", os.path.join(ROOT, "examples", "fp8_moe_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    _, _, far = example.run(tokens, channels, hidden, experts, top, vocab)
    # e4m3 keeps 4 significant bits: a value is off by 2^-4 / sqrt(3) = 3.6 % of
    # itself at most on average, a product of two by 5 %, and the block chains
    # two products (7 %) and for the logits a third (9 %); doubled.
    assert far["h"] < 0.14 and far["logits"] < 0.18, far
