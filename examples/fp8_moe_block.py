"""An expert feed-forward block in 8-bit floating point, with the library's
operators used together as in serving:

  residual stream --norm_residual--> block input
    --route_topk--> experts and weights of each token
    --dispatch_rows(quantize)--> codes + row scales by expert, offsets on the device
    --gemm_fp8_grouped--> gate and up --silu * mul, quantize_fp8-->
    --gemm_fp8_grouped--> down --combine_rows--> block output
    --norm_residual--> next residual stream and next block's input
    --gemm_fp8--> logits of the last token

Nothing is copied to the host between the first norm and the logits.

    python examples/fp8_moe_block.py [--tokens 512] [--channels 2048] [--hidden 1024]
                                     [--experts 16] [--top 2] [--vocab 8192]

prints how far the block is from the same block in 32 bits and its time.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tma_pipelined_tensor_tn_gb300 as tg  # noqa: E402


class Block:
    """Weights of one block, quantised once per 128 x 128 values."""

    def __init__(self, channels, hidden, experts, vocab, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, fan_in):
            return torch.randn(shape, device="cuda", generator=g) * fan_in ** -0.5

        self.w_pre = torch.ones(channels, device="cuda", dtype=torch.bfloat16)
        self.w_post = torch.ones_like(self.w_pre)
        self.w_next = torch.ones_like(self.w_pre)
        self.router = weight(experts, channels, fan_in=channels).bfloat16()
        self.up = weight(experts, 2 * hidden, channels, fan_in=channels).bfloat16()
        self.down = weight(experts, channels, hidden, fan_in=hidden).bfloat16()
        self.head = weight(vocab, channels, fan_in=channels).bfloat16()
        self.experts = experts
        self.first = torch.arange(experts + 1, device="cuda")
        # Whole matrices of experts share the 128-row blocks when their rows are
        # a multiple of 128; each is quantised by itself to allow any size.
        self.up_q, self.up_s = self._stack(self.up)
        self.down_q, self.down_s = self._stack(self.down)
        self.head_q, self.head_s = tg.quantize_fp8(self.head, block_rows=128)

    @staticmethod
    def _stack(w):
        pairs = [tg.quantize_fp8(m, block_rows=128) for m in w]
        return torch.stack([q.view(torch.uint8) for q, _ in pairs]).view(torch.float8_e4m3fn), \
            torch.stack([s for _, s in pairs])

    def route(self, x, top):
        """The plain block's routing: source rows sorted by expert, their weights, and the
        experts' row offsets."""
        p, expert = torch.topk(torch.softmax((x @ self.router.t()).float(), dim=1), top)
        expert, order = torch.sort(expert.flatten(), stable=True)
        # First row of each expert (torch.bincount would wait for the device).
        offsets = torch.searchsorted(expert, self.first, out_int32=True)
        return order // top, (p / p.sum(1, keepdim=True)).flatten()[order], offsets

    def __call__(self, h, top):
        """(next residual stream, next block's input, logits of the last token)."""
        # The router reads the 16-bit norm, the experts its codes.
        x = tg.norm_residual(h, w_pre=self.w_pre).x
        ids, share = tg.route_topk(x @ self.router.t(), top)
        r = tg.dispatch_rows(x, ids, self.experts, quantize=True)
        gate, up = tg.gemm_fp8_grouped(r.rows, r.scales, self.up_q, self.up_s,
                                       r.offsets).chunk(2, dim=1)
        act, act_s = tg.quantize_fp8(torch.nn.functional.silu(gate) * up)
        out = tg.gemm_fp8_grouped(act, act_s, self.down_q, self.down_s, r.offsets)
        y = tg.combine_rows(out, r.row_of, share)
        n = tg.norm_residual(h, y, w_post=self.w_post, w_pre=self.w_next, quantize=True)
        logits = tg.gemm_fp8(n.x[-1:], n.scales[-1:], self.head_q, self.head_s)
        return n.h, n.x, logits

    def plain(self, h, top):
        """The same block with 16-bit weights in 32-bit arithmetic."""
        def norm(v, w):
            return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6) * w.float()

        x = norm(h.float(), self.w_pre)
        rows, share, offsets = self.route(x.to(h.dtype), top)
        y = torch.zeros_like(x)
        for e, (lo, hi) in enumerate(zip(offsets[:-1].tolist(), offsets[1:].tolist())):
            gate, up = (x[rows[lo:hi]] @ self.up[e].float().t()).chunk(2, dim=1)
            out = (torch.nn.functional.silu(gate) * up) @ self.down[e].float().t()
            y.index_add_(0, rows[lo:hi], out * share[lo:hi, None])
        h2 = h.float() + norm(y, self.w_post)
        x2 = norm(h2, self.w_next)
        return h2, x2, x2[-1:] @ self.head.float().t()


def run(tokens, channels, hidden, experts, top, vocab, seed=0):
    """Relative distances of the block's results from the plain block's."""
    block = Block(channels, hidden, experts, vocab, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    h = torch.randn((tokens, channels), device="cuda", generator=g).bfloat16()
    got, want = block(h, top), block.plain(h, top)
    tg.check()
    far = {}
    for name, a, b in zip(("h", "x", "logits"), got, want):
        if name == "x":     # codes: what they stand for is seen in the logits
            continue
        far[name] = float((a.float() - b).norm() / b.norm())
    return block, h, far


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 512), ("channels", 2048), ("hidden", 1024), ("experts", 16),
                        ("top", 2), ("vocab", 8192)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    block, h, far = run(a.tokens, a.channels, a.hidden, a.experts, a.top, a.vocab)
    print("relative distance from the 32-bit block:", far)
    for _ in range(10):
        block(h, a.top)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(50):
        block(h, a.top)
    end.record()
    torch.cuda.synchronize()
    print(f"{start.elapsed_time(end) / 50 * 1e3:.1f} us per block of {a.tokens} tokens")


if __name__ == "__main__":
    main()
