"""Drafted trees and beams on the decoder block's operators: every step checks a tree of drafted tokens
per sequence at once and keeps one path of it; now and then the sequences are beams that branch.

    python examples/draft_trees.py [--batch 16] [--prompt 300] [--steps 32]

The block of decode_block.py (width 256, 4 query and 2 key/value heads of 64, paged e4m3 cache).  A step:

    pages     cache_pages           room for the drafts; pages of lost tokens and ended rows come back
    copies    cache_copy            pages that branched rows write on
    append    rotary, cache_append  keys and queries turned by the nodes' depths, all nodes cached
    attention cache_tree_attention  each node over the older tokens and its ancestors
    keep      cache_compact         the accepted path's tokens moved together

Nothing of a step waits for the host.  Weights and drafts are random (seeded): a node is accepted where a
fixed projection of its output prefers it among its siblings and is not below zero.
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from examples.decode_block import HEAD, HEADS, KV_HEADS, PAGE, WIDTH, DecoderBlock     # noqa: E402
from gemm_conv_chains_gb300 import ops                                               # noqa: E402

# A tree of 10 drafted tokens behind the last accepted one (node 0), three levels.
PARENTS = [-1, 0, 0, 0, 1, 1, 2, 3, 4, 4, 6]
NODES = len(PARENTS)
DEPTH = [0] * NODES
for _i, _p in enumerate(PARENTS):
    DEPTH[_i] = DEPTH[_p] + 1 if _p >= 0 else 0
LEVELS = max(DEPTH)
FAN = max(PARENTS.count(i) for i in range(NODES))


def masks():
    """[NODES, 1] int64: each node's ancestors and itself."""
    seen = []
    for i, p in enumerate(PARENTS):
        seen.append((seen[p] if p >= 0 else 0) | 1 << i)
    return torch.tensor(seen, dtype=torch.int64)[:, None]


class Rows:
    """The cache and the page table of its sequences, all on the GPU; two tables taken in turn."""

    def __init__(self, batch, pages, width):
        shape = (pages, KV_HEADS, PAGE, HEAD)
        self.k = torch.zeros(shape, device="cuda").to(torch.float8_e4m3fn)
        self.v = torch.zeros_like(self.k)
        self.k_scale = torch.zeros(pages, KV_HEADS, device="cuda")
        self.v_scale = torch.zeros_like(self.k_scale)
        self.pages = pages
        self.tables = [self._out(batch, width) for _ in range(2)]
        self.table, self.lens = self.tables[0][:2]
        self.table.fill_(-1)
        self.lens.zero_()
        self.left = None

    def _out(self, rows, width):
        def ints(*shape):
            return torch.empty(shape, dtype=torch.int32, device="cuda")
        return ints(rows, width), ints(rows), ints(rows, 3), ints(1)

    def pool(self):
        return self.k, self.v, self.k_scale, self.v_scale

    def step(self, new, kept=None, parents=None):
        """Rows that follow `parents` (None: each itself) for `kept` tokens (None: all) with room for
        new[b] more; pages that several rows write on are copied."""
        out = self.tables[1] if self.table is self.tables[0][0] else self.tables[0]
        self.table, self.lens, copies, self.left = ops.cache_pages(
            self.table, self.lens, self.pages, PAGE, parents, kept, new, out=out)
        ops.cache_copy(*self.pool(), copies)


class TreeBlock(DecoderBlock):
    """The decoder block over drafted trees."""

    def __init__(self, batch, **kw):
        super().__init__(**kw)
        self.masks = masks().repeat(batch, 1).cuda()
        self.depth = torch.tensor(DEPTH, dtype=torch.int32, device="cuda")
        children = [[j for j in range(NODES) if PARENTS[j] == i] for i in range(NODES)]
        self.children = torch.tensor([c + [-1] * (FAN - len(c)) for c in children], device="cuda")
        g = torch.Generator().manual_seed(7)
        self.prefer = torch.randn(WIDTH, generator=g).cuda()

    def prompts(self, x, rows, new, most):
        """x [sum(new), 256]: prompts, as decode_block's block takes them."""
        starts = torch.nn.functional.pad(new.cumsum(0), (1, 0)).to(torch.int32)
        rows.step(new)
        pool = (*rows.pool(), rows.table, rows.lens, starts, most)
        T = x.shape[0]
        q = ops.gemm_bias_act(x, self.wq, None, "none").view(T, HEADS, HEAD)
        kv = ops.gemm_bias_act(x, self.wkv, None, "none").view(T, 2 * KV_HEADS, HEAD)
        q = ops.cache_append(kv[:, :KV_HEADS], kv[:, KV_HEADS:], *pool, table=self.table, q=q, q_out=q)
        return self._rest(x, ops.cache_attention(q, *pool))

    def _rest(self, x, a):
        x = x + ops.gemm_bias_act(a.view(x.shape[0], HEADS * HEAD), self.wo, None, "none")
        return x + ops.b2b_gemm(x, self.w0, None, self.w1, None, "hardswish", "none")

    def drafts(self, x, rows):
        """x [batch * NODES, 256]: every node's input; the rows have room for them."""
        T, batch = x.shape[0], x.shape[0] // NODES
        first = rows.lens - NODES
        positions = (first[:, None] + self.depth).flatten()
        q = ops.gemm_bias_act(x, self.wq, None, "none").view(T, HEADS, HEAD)
        kv = ops.gemm_bias_act(x, self.wkv, None, "none").view(T, 2 * KV_HEADS, HEAD)
        q = ops.rotary(q, self.table, positions, out=q)
        k = ops.rotary(kv[:, :KV_HEADS], self.table, positions, out=kv[:, :KV_HEADS])
        pool = (*rows.pool(), rows.table, rows.lens)
        ops.cache_append(k, kv[:, KV_HEADS:], *pool)
        a = ops.cache_tree_attention(q, self.masks[:T], *pool, positions=positions)
        return self._rest(x, a).view(batch, NODES, WIDTH)

    def accept(self, y):
        """(path [batch, LEVELS + 1], count [batch]): from node 0 down the preferred children."""
        batch = y.shape[0]
        score = y.float() @ self.prefer
        node = torch.zeros(batch, dtype=torch.long, device="cuda")
        going = torch.ones(batch, dtype=torch.bool, device="cuda")
        count = torch.ones(batch, dtype=torch.int32, device="cuda")
        path = [node]
        for _ in range(LEVELS):
            child = self.children[node]
            s = score.gather(1, child.clamp_min(0)).masked_fill(child < 0, -math.inf)
            best, at = s.max(-1)
            going = going & (best >= 0)
            node = torch.where(going, child.gather(1, at[:, None])[:, 0], node)
            count += going.to(torch.int32)
            path.append(node)
        return torch.stack(path, 1), count

    def keep(self, rows, path, count):
        """The accepted tokens moved together; the lengths after."""
        first = rows.lens - NODES
        ops.cache_compact(*rows.pool(), rows.table, rows.lens, first,
                          (first[:, None] + path).to(torch.int32), count)
        return first + count


def branch(batch):
    """Beams of four: the last of each four branches off the first."""
    parents = torch.arange(batch, dtype=torch.int32)
    parents[3::4] = parents[0::4][: parents[3::4].numel()]
    return parents.cuda()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=300, help="the longest prompt")
    ap.add_argument("--steps", type=int, default=32)
    args = ap.parse_args()
    B = args.batch
    new = [1 + (args.prompt - 1) * (b + 1) // B for b in range(B)]
    most = max(new) + (args.steps + 3) * (LEVELS + 1) + NODES
    width = -(-most // PAGE)
    block = TreeBlock(B, positions=most)
    rows = Rows(B, 2 * B * width, width)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(sum(new), WIDTH, generator=g, device="cuda").bfloat16()
    y = block.prompts(x, rows, torch.tensor(new, dtype=torch.int32, device="cuda"), max(new))
    last = y[torch.tensor(new, device="cuda").cumsum(0) - 1]
    room = torch.full((B,), NODES, dtype=torch.int32, device="cuda")
    parents, kept, accepted = branch(B), rows.lens.clone(), torch.zeros(B, dtype=torch.int32, device="cuda")
    for step in range(3 + args.steps):
        if step == 3:
            torch.cuda.synchronize()
            t0, accepted = time.perf_counter(), accepted * 0
        branches = step % 4 == 3
        if branches:
            kept, last = kept[parents.long()], last[parents.long()]
        rows.step(room, kept, parents if branches else None)
        drafted = torch.randn(B, NODES, WIDTH, generator=g, device="cuda").bfloat16()
        drafted[:, 0] = last / last.float().square().mean(-1, keepdim=True).sqrt().to(last.dtype)
        y = block.drafts(drafted.view(B * NODES, WIDTH), rows)
        path, count = block.accept(y)
        kept = block.keep(rows, path, count)
        last = y.gather(1, path[:, -1, None, None].expand(B, 1, WIDTH))[:, 0]
        accepted += count
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) / args.steps * 1e3
    st, info = ops.get_cache_error()
    assert st == 0, f"cache error {info}"
    assert rows.left.item() >= 0
    per = accepted.sum().item() / (args.steps * B)
    print(f"{sum(new)} prompt tokens, then trees of {NODES} nodes on {B} sequences: {ms:.3f} ms per step, "
          f"{per:.2f} of {LEVELS + 1} tokens kept, {per * B / ms * 1e3:.0f} tokens/s; "
          f"{rows.left.item()} of {rows.pages} pages free; |x| = {last.float().norm().item():.3f}")


if __name__ == "__main__":
    main()
