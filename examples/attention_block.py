"""One attention block with 4-bit linears and a 4-bit key-value cache: prompts
of several sequences in one call, then a token at a time.

    python examples/attention_block.py

The linears are W4A4 (quantize + gemm); keys and values go to the cache as
they are rotated (kv_append), and the queries read it there (kv_attention).
A step's tokens lie behind one another whatever their sequences; where their
rows are kept and how long each sequence is, the host decides (Sequences).
"""
import sys
import time
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
import block_scaled_fp4_amax_amd as fp4  # noqa: E402


class Sequences:
    """Which pages hold which sequence: pages are taken as sequences grow and
    given back when they end."""

    def __init__(self, num_pages, page_size, batch, max_len):
        self.page_size = page_size
        self.free = list(range(num_pages))[::-1]
        self.pages = [[] for _ in range(batch)]
        self.lens = [0] * batch
        self.table = torch.full((batch, -(-max_len // page_size)), -1, dtype=torch.int32)

    def step(self, counts):
        """Make room for counts[b] more tokens of each sequence. Returns what
        kv_append and kv_attention need to know of the step, on the GPU."""
        slots, positions, offsets = [], [], [0]
        for b, n in enumerate(counts):
            for at in range(self.lens[b], self.lens[b] + n):
                if at % self.page_size == 0:
                    self.table[b, len(self.pages[b])] = self.free[-1]
                    self.pages[b].append(self.free.pop())
                slots.append(self.pages[b][-1] * self.page_size + at % self.page_size)
                positions.append(at)
            self.lens[b] += n
            offsets.append(offsets[-1] + n)
        single = all(n == 1 for n in counts)
        return dict(slots=torch.tensor(slots).cuda(), positions=torch.tensor(positions).cuda(),
                    table=self.table.cuda(), lens=torch.tensor(self.lens, dtype=torch.int32).cuda(),
                    offsets=None if single else torch.tensor(offsets, dtype=torch.int32).cuda(),
                    max_len=max(self.lens))

    def end(self, b):
        self.free += self.pages[b][::-1]
        self.pages[b], self.lens[b] = [], 0
        self.table[b] = -1


class AttentionBlock:
    """out = W_o attention(W_qkv x) with rotary positions, all weights random."""

    def __init__(self, hidden, heads, kv_heads, head_dim, cache, max_positions, seed=0):
        self.heads, self.kv_heads, self.dim, self.cache = heads, kv_heads, head_dim, cache
        g = torch.Generator().manual_seed(seed)

        def weight(n, k):
            return fp4.quantize((torch.randn(n, k, generator=g) * k ** -0.5).bfloat16().cuda(), "nvfp4",
                                four_over_six=True)
        self.w_qkv = weight((heads + 2 * kv_heads) * head_dim, hidden)
        self.w_o = weight(hidden, heads * head_dim)
        angle = torch.arange(max_positions)[:, None] / 10000.0 ** (torch.arange(0, head_dim, 2) / head_dim)
        self.cos, self.sin = angle.cos().cuda(), angle.sin().cuda()

    def linear(self, x, w):
        return fp4.gemm(fp4.quantize(x, "nvfp4", four_over_six=True), w, torch.bfloat16)

    def attend(self, x, step):
        """x [tokens, hidden]: the rotated queries and what attention makes of them."""
        qkv = self.linear(x, self.w_qkv).view(len(x), -1, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)  # rows with strides, never copied
        q = fp4.kv_append(self.cache, k, v, step["slots"], q=q, positions=step["positions"], cos=self.cos,
                          sin=self.sin, four_over_six=self.cache.fmt == fp4.FP4_NVFP4)
        return q, fp4.kv_attention(q, self.cache, step["table"], step["lens"], q_offsets=step["offsets"],
                                   max_kv_len=step["max_len"])

    def __call__(self, x, step):
        return self.linear(self.attend(x, step)[1].flatten(1), self.w_o)


def main(fmt="nvfp4", hidden=4096, heads=32, kv_heads=8, head_dim=128, prompts=(1000, 37, 512, 2048), tokens=32):
    batch, page_size, longest = len(prompts), 64, max(prompts) + tokens
    pages = sum(-(-(n + tokens) // page_size) for n in prompts)
    cache = fp4.KVCache.empty(fmt, pages, page_size, kv_heads, head_dim, k_amax=16.0, v_amax=16.0, four_over_six=True)
    seqs = Sequences(pages, page_size, batch, longest)
    block = AttentionBlock(hidden, heads, kv_heads, head_dim, cache, longest)

    def run(counts):
        step = seqs.step(counts)
        x = torch.randn(sum(counts), hidden, device="cuda", dtype=torch.bfloat16)
        torch.cuda.synchronize()
        t = time.perf_counter()
        y = block(x, step)
        torch.cuda.synchronize()
        return y, (time.perf_counter() - t) * 1e6

    y, us = run(prompts)
    print(f"prompts of {prompts}: {tuple(y.shape)} in {us:.0f} us (with what the first call loads)")
    times = [run([1] * batch)[1] for _ in range(tokens)]
    held = sum(t.numel() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales))
    plain = 4 * pages * page_size * kv_heads * head_dim
    print(f"{tokens} tokens of each: {sorted(times)[tokens // 2]:.0f} us a step (median)")
    print(f"cache: {held / 2**20:.1f} MiB ({plain / 2**20:.1f} in bf16)")


if __name__ == "__main__":
    main()
