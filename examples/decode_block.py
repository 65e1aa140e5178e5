"""A decoder block on the framework's operators: prompts in, then tokens one by one.

    python examples/decode_block.py [--batch 16] [--prompt 300] [--steps 64]

Width 256: 4 query and 2 key/value heads of 64, half layout rotary positions, a paged e4m3 cache,
and the fused FFN chain 256 -> 256 -> 256.  Per call, whatever the number of new tokens:

    q, kv     gemm_bias_act x 2
    cache     cache_append       keys and queries rotated, keys and values quantised, in one launch
    attention cache_attention    causal over each sequence's pages
    output    gemm_bias_act, then b2b_gemm (both GEMMs of the FFN in one kernel)

Weights are random (seeded); the residual additions are torch's.
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gemm_conv_chains_gb300 import ops                                     # noqa: E402

WIDTH, HEADS, KV_HEADS, HEAD, PAGE = 256, 4, 2, 64, 32
WARMUP = 3                                                # untimed steps


class Pages:
    """The block's cache pools and the page lists of its sequences (a free list, nothing evicted).
    The host keeps the lengths; the GPU's copies change only where they have to."""

    def __init__(self, batch, pages, max_pages):
        shape = (pages, KV_HEADS, PAGE, HEAD)
        self.k = torch.zeros(shape, device="cuda").to(torch.float8_e4m3fn)
        self.v = torch.zeros_like(self.k)
        self.k_scale = torch.zeros(pages, KV_HEADS, device="cuda")
        self.v_scale = torch.zeros_like(self.k_scale)
        self.table = torch.full((batch, max_pages), -1, dtype=torch.int32)
        self.table_gpu = self.table.cuda()
        self.lens = [0] * batch
        self.lens_gpu = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.free = list(range(pages))
        self.new, self.new_gpu, self.starts_gpu = None, None, None

    def grow(self, new):
        """Makes room for new[b] more tokens; the calls' arguments (table, lens, starts)."""
        if new != self.new:
            self.new, self.new_gpu = new, torch.tensor(new, dtype=torch.int32, device="cuda")
            self.starts_gpu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
        grown = False
        for b, n in enumerate(new):
            have = -(-self.lens[b] // PAGE)
            self.lens[b] += n
            for j in range(have, -(-self.lens[b] // PAGE)):
                self.table[b, j] = self.free.pop()
                grown = True
        if grown:
            self.table_gpu = self.table.cuda()
        self.lens_gpu = self.lens_gpu + self.new_gpu
        return self.table_gpu, self.lens_gpu, self.starts_gpu


class DecoderBlock:
    def __init__(self, dtype=torch.bfloat16, positions=4096, seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(k, n):
            return (torch.randn(k, n, generator=g) / math.sqrt(k)).to(dtype).cuda()

        self.wq, self.wkv = weight(WIDTH, HEADS * HEAD), weight(WIDTH, 2 * KV_HEADS * HEAD)
        self.wo = weight(HEADS * HEAD, WIDTH)
        self.w0, self.w1 = weight(WIDTH, WIDTH), weight(WIDTH, WIDTH)
        self.table = ops.rotary_table(positions, HEAD)

    def __call__(self, x, cache, new):
        """x [sum(new), 256]: the new tokens' rows, sequence after sequence."""
        page_table, lens, starts = cache.grow(new)
        T, most = x.shape[0], max(new)
        q = ops.gemm_bias_act(x, self.wq, None, "none").view(T, HEADS, HEAD)
        kv = ops.gemm_bias_act(x, self.wkv, None, "none").view(T, 2 * KV_HEADS, HEAD)
        pool = (cache.k, cache.v, cache.k_scale, cache.v_scale, page_table, lens, starts, most)
        q = ops.cache_append(kv[:, :KV_HEADS], kv[:, KV_HEADS:], *pool, table=self.table, q=q, q_out=q)
        a = ops.cache_attention(q, *pool)
        x = x + ops.gemm_bias_act(a.view(T, HEADS * HEAD), self.wo, None, "none")
        return x + ops.b2b_gemm(x, self.w0, None, self.w1, None, "hardswish", "none")


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=300, help="the longest prompt")
    ap.add_argument("--steps", type=int, default=64)
    args = ap.parse_args()
    new = [1 + (args.prompt - 1) * (b + 1) // args.batch for b in range(args.batch)]
    most = max(new) + WARMUP + args.steps
    per_seq = -(-most // PAGE)
    block = DecoderBlock(positions=most)
    cache = Pages(args.batch, args.batch * per_seq, per_seq)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(sum(new), WIDTH, generator=g, device="cuda").bfloat16()
    y = block(x, cache, new)                                  # the prompts, ragged
    one = [1] * args.batch
    last = torch.tensor(new, device="cuda").cumsum(0) - 1
    x = y[last]
    for step in range(WARMUP + args.steps):
        if step == WARMUP:
            torch.cuda.synchronize()
            t0 = time.perf_counter()
        x = block(x / x.float().square().mean(-1, keepdim=True).sqrt().to(x.dtype), cache, one)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) / args.steps * 1e3
    st, info = ops.get_cache_error()
    assert st == 0, f"cache error {info}"
    print(f"{sum(new)} prompt tokens, then steps of {args.batch} sequences: "
          f"{ms:.3f} ms per step, {args.batch / ms * 1e3:.0f} tokens/s; cached "
          f"{sum(cache.lens)} tokens in {(cache.table >= 0).sum().item()} pages; "
          f"|x| = {x.float().norm().item():.3f}")


if __name__ == "__main__":
    main()
