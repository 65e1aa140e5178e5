"""Plain forms of the operators of drafted and branching sequences, for their tests (not collected)."""
import math
import random

import torch

from decoder_ref import F8


def tree(n, seed, spread=4):
    """Parents of n nodes: node 0 a root, the others under one of the last few."""
    r = random.Random(seed)
    return [-1] + [r.randint(max(0, i - spread), i - 1) for i in range(1, n)]


def ancestors(parents):
    """[n, n] bool: who is an ancestor of whom, itself counted."""
    n = len(parents)
    seen = torch.zeros(n, n, dtype=torch.bool)
    for i, p in enumerate(parents):
        if p >= 0:
            seen[i] = seen[p]
        seen[i, i] = True
    return seen


def words(blocks, width=None):
    """The masks of the sequences' [n, n] blocks, int64 [T, width]."""
    width = width or max(1, -(-max(s.shape[0] for s in blocks) // 64))
    out = []
    for s in blocks:
        for row in s.tolist():
            m = sum(1 << j for j, b in enumerate(row) if b)
            out.append([((m >> 64 * w) & (1 << 64) - 1) for w in range(width)])
    return torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in out],
                        dtype=torch.int64).reshape(-1, width)


def tree_attention(cache, q, blocks, scale, softcap=0.0, slopes=None, positions=None):
    """(out, allowed error before the output's rounding), float64 [T, q heads, D]: as
    decoder_ref.attention, with blocks[b] [n, n] saying which new tokens a row sees."""
    T, Hq, D = q.shape
    group = Hq // cache.heads
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    at = 0
    for b, n in enumerate(cache.new):
        if n == 0:
            continue
        length = cache.lens[b]
        k, v = cache.values(b, length)
        seen = torch.cat([torch.ones(n, length - n, dtype=torch.bool), blocks[b]], 1)
        mine = torch.arange(length - n, length) if positions is None else positions[at: at + n].long()
        keys = torch.cat([torch.arange(length - n), mine])
        for h in range(Hq):
            qh, kh, vh = q[at: at + n, h].double(), k[h // group], v[h // group]
            z = qh @ kh.T * scale
            # fp32 sums of D products in any order, the factors and the exponent's own rounding
            size = qh.abs() @ kh.abs().T * abs(scale)
            if softcap:
                z = softcap * torch.tanh(z / softcap)
                size = size + 8 * softcap
            if slopes is not None:
                bias = slopes[h].double() * (keys - mine[:, None])
                z = z + bias
                size = size + bias.abs()
            delta = (D + 16) * 2.0 ** -24 * size
            # (a row that sees nothing has no largest score: its weights are zeros)
            z = torch.where(seen, z, -math.inf)
            e = torch.exp(z - z.amax(-1, keepdim=True).clamp_min(-1e30))     # (of a NaN: all NaN)
            p = torch.where(seen, e, 0) / e.sum(-1, keepdim=True).clamp_min(1e-300)
            # what a row does not see does not enter it, a NaN neither
            vs = torch.where(seen.any(0)[:, None], vh, 0)
            one = torch.stack([p[i, seen[i]] @ vh[seen[i]] for i in range(n)])
            # (NaN scores and codes make NaN outputs; the others' bounds are what counts)
            p, delta = torch.nan_to_num(p), torch.nan_to_num(delta)
            mag = torch.where(seen, p * (2.0 ** -11 + 2.0 ** -18 + 2 * delta), 0)
            clean = torch.nan_to_num(vs.abs())
            out[at: at + n, h] = one
            tol[at: at + n, h] = mag @ clean + torch.where(seen, p * delta, 0).sum(-1, keepdim=True) * (p @ clean)
            # fp16 below its normal range: 2^-25 of the largest scale's power of two per token,
            # relative to the largest probability
            top = p.max(-1, keepdim=True).values
            tol[at: at + n, h] += top * length * 2.0 ** -25 * 2 * clean.max()
        at += n
    return out, tol


def pages(table, lens, pages, page, parents=None, kept=None, new=None):
    """(table, lens, copies, left) of the rows that follow, by lists, row after row."""
    width = len(table[0]) if table else 0
    rows = len(parents) if parents is not None else len(table)
    parents = list(range(rows)) if parents is None else parents
    kept = [lens[p] if p >= 0 else 0 for p in parents] if kept is None else kept
    new = [0] * rows if new is None else new
    held = []                                        # each row's old pages
    for p, k in zip(parents, kept):
        held.append(list(table[p][: -(-k // page)]) if p >= 0 else [])
    writers, readers = {}, set()
    for r in range(rows):
        for j, x in enumerate(held[r]):
            if new[r] > 0 and kept[r] % page and j == len(held[r]) - 1:
                writers.setdefault(x, []).append(r)
            else:
                readers.add(x)
    used = set(writers) | readers
    free = [x for x in range(pages) if x not in used]
    out, copies, short = [], [], 0

    def take():
        nonlocal short
        if free:
            return free.pop(0)
        short += 1
        return -1

    for r in range(rows):
        mine, copy = held[r], [-1, -1, 0]
        if new[r] > 0 and kept[r] % page:
            x = mine[-1]
            if x in readers or writers[x][0] != r:
                mine[-1] = take()
                if mine[-1] >= 0:
                    copy = [x, mine[-1], kept[r] % page]
        while len(mine) < -(-(kept[r] + new[r]) // page):
            mine.append(take())
        out.append(mine + [-1] * (width - len(mine)))
        copies.append(copy)
    return out, [k + n for k, n in zip(kept, new)], copies, [len(free) - short]


def compact(codes, scale, table, page, first, tokens, counts):
    """One pool after its sequences' kept tokens are moved together: (codes, scale, allowed error of
    each value), float64 values of codes."""
    old, had = codes.double(), scale.double()
    now, s_now = old.clone(), had.clone()
    for b, (f, n) in enumerate(zip(first, counts)):
        if n == 0:
            continue
        come = list(range(f // page * page, f)) + list(tokens[b][:n])
        for j in range(0, len(come), page):
            at = int(table[b][f // page + j // page])
            part = come[j: j + page]
            ids = torch.tensor([int(table[b][c // page]) for c in part])
            slots = torch.tensor([c % page for c in part])
            s = had[ids]                                             # [tokens, heads]
            top = s.amax(0)
            ratio = torch.where(s == top, 1.0, (s.float() / top.float()).double())
            # codes times the ratio in fp32, then half a step: the same two roundings
            v = (old[ids, :, slots].float() * ratio.float()[..., None]).to(F8).double()
            now[at, :, : len(part)] = v.transpose(0, 1)
            s_now[at] = top
    return now, s_now
