"""The example that uses the 8-bit operators together, at small odd sizes."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    import tma_pipelined_tensor_tn_gb300 as tg
    tg.build()
    spec = importlib.util.spec_from_file_location(
        "fp8_moe_block", os.path.join(ROOT, "examples", "fp8_moe_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


def test_fp8_block_never_waits_for_the_device():
    """Nothing is copied to the host: the block runs with synchronising calls turned
    into errors, and is captured in a graph that follows its input."""
    block = load().Block(512, 256, 8, 1000)
    h = torch.randn((77, 512), device="cuda").bfloat16()
    want = block(h, 2)
    torch.cuda.synchronize()
    before = torch.cuda.get_sync_debug_mode()
    torch.cuda.set_sync_debug_mode("error")
    try:
        block(h, 2)
    finally:
        torch.cuda.set_sync_debug_mode(before)
    torch.cuda.synchronize()
    other = torch.randn_like(h)
    h0, h = h.clone(), other
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(h, 2)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(h, 2)
    h.copy_(h0)
    graph.replay()
    torch.cuda.synchronize()
    # Two experts a token: their sum is the same in either order.
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert torch.equal(got[1].view(torch.uint8), want[1].view(torch.uint8))


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
