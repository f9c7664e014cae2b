"""A mixture-of-experts layer with 4-bit experts: a prompt through the grouped
W4A4 products, then a few tokens at a time through products of their rows.

    python examples/moe_layer.py

The router chooses (moe_route). A prompt's tokens are quantized once, carried
to their experts packed (moe_group, moe_dispatch), multiplied (gemm_grouped)
and brought back (moe_combine). A step of few tokens reads each expert's
weights once, in 4 bits, against activations in bf16 (matvec).
"""
import sys
import time
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
import block_scaled_fp4_amax_amd as fp4  # noqa: E402


class MoeLayer:
    """out = sum_j w_j W2_e (silu(W1_e x) * W3_e x) over each token's top_k experts e; all weights random."""

    def __init__(self, hidden, inter, experts, top_k, fmt="mxfp4", score="softmax", seed=0):
        self.experts, self.top_k, self.fmt, self.score = experts, top_k, fmt, score
        g = torch.Generator().manual_seed(seed)

        def weight(n, k):
            return fp4.quantize((torch.randn(experts, n, k, generator=g) * k ** -0.5).bfloat16().cuda(), fmt,
                                four_over_six=True)
        self.w13, self.w2 = weight(2 * inter, hidden), weight(hidden, inter)  # W1 and W3 in one
        self.router = (torch.randn(experts, hidden, generator=g) * hidden ** -0.5).cuda()
        self.bias = torch.zeros(experts, device="cuda") if score == "sigmoid" else None  # balances the load

    def route(self, x):
        return fp4.moe_route(x.float() @ self.router.T, self.top_k, score=self.score, bias=self.bias)

    def gate(self, h):
        a, b = h.chunk(2, -1)
        return torch.nn.functional.silu(a) * b

    def few(self, x):
        w, ids = self.route(x)
        h = self.gate(fp4.matvec(x, self.w13, ids))
        return fp4.moe_combine(fp4.matvec(h, self.w2, ids), w)

    def many(self, x):
        w, ids = self.route(x)
        groups = fp4.moe_group(ids, self.experts)
        rows = fp4.moe_dispatch(fp4.quantize(x, self.fmt, four_over_six=True), groups)
        h = self.gate(fp4.gemm_grouped(rows, self.w13, groups.offsets, torch.bfloat16))
        y = fp4.gemm_grouped(fp4.quantize(h, self.fmt, four_over_six=True), self.w2, groups.offsets, torch.bfloat16)
        return fp4.moe_combine(y, w, groups)

    def __call__(self, x):
        # few rows an expert: the weights' bytes are the work, and they are read once either way
        return self.few(x) if len(x) * self.top_k <= 4 * self.experts else self.many(x)


def main(fmt="mxfp4", hidden=2880, inter=2880, experts=32, top_k=4, prompt=2048, batch=8, steps=32):
    layer = MoeLayer(hidden, inter, experts, top_k, fmt)

    def run(tokens):
        x = torch.randn(tokens, hidden, device="cuda", dtype=torch.bfloat16)
        torch.cuda.synchronize()
        t = time.perf_counter()
        y = layer(x)
        torch.cuda.synchronize()
        return y, (time.perf_counter() - t) * 1e6

    y, us = run(prompt)
    print(f"prompt of {prompt}: {tuple(y.shape)} in {us:.0f} us (with what the first call loads)")
    times = [run(batch)[1] for _ in range(steps)]
    print(f"{batch} tokens: {sorted(times)[steps // 2]:.0f} us a step (median)")


if __name__ == "__main__":
    main()
