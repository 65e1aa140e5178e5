"""Plain 64-bit forms of the decoder-block operators, for their tests (not collected)."""
import math

import torch

F8 = torch.float8_e4m3fn
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}      # half a step, relative
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}    # and below the normal range


def table64(n, rot, base=10000.0):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1)


def turn(x, cs, layout, inverse=False):
    """x [T, H, D] float64, cs [T, rot / 2, 2]."""
    half = cs.shape[1]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1] * (-1 if inverse else 1)
    y = x.clone()
    if layout == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    return y


class Cache:
    """A random cache over sequences of the given older and new token counts, on the CPU."""

    def __init__(self, older, new, heads, D, page, seed=0, spare=3, fill=None):
        g = torch.Generator().manual_seed(seed)
        self.older, self.new, self.page, self.heads, self.D = older, new, page, heads, D
        self.lens = [a + n for a, n in zip(older, new)]
        need = [-(-n // page) for n in self.lens]
        self.pages = sum(need) + spare
        shape = (self.pages, heads, page, D)
        self.k = (torch.randn(shape, generator=g) * 40).to(F8)
        self.v = (torch.randn(shape, generator=g) * 40).to(F8)
        self.ks = torch.rand(self.pages, heads, generator=g) * 0.03 + 0.01
        self.vs = torch.exp(torch.randn(self.pages, heads, generator=g)) * 0.01
        order = torch.randperm(self.pages, generator=g).tolist()
        self.table = torch.full((len(older), max(need + [1]) + 1), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
        self.starts = torch.tensor([0] + new).cumsum(0).to(torch.int32)
        self.T = sum(new)
        if fill is not None:                        # whatever no token has been written to
            used = torch.zeros(self.pages, page, dtype=torch.bool)
            for b, n in enumerate(self.lens):
                for j in range(n):
                    used[self.table[b, j // page], j % page] = True
            raw = ~used[:, None, :, None].expand(shape)
            for t in (self.k, self.v):
                t.view(torch.uint8)[raw] = fill
            lone = ~used.any(1)
            self.ks[lone] = math.nan
            self.vs[lone] = math.nan

    def args(self, starts=True, max_new=True):
        """The entry points' cache arguments, on the GPU."""
        self.dev = [t.cuda() for t in (self.k, self.v, self.ks, self.vs, self.table,
                                       torch.tensor(self.lens, dtype=torch.int32))]
        if starts:
            self.dev.append(self.starts.cuda())
            if max_new:
                self.dev.append(max(self.new))
        return self.dev

    def values(self, b, n):
        """k, v [heads, n, D] float64 of sequence b's first n tokens."""
        ids = self.table[b, : -(-n // self.page)].long()
        return tuple((c.double()[ids] * s[ids].double()[..., None, None]).transpose(0, 1).reshape(
            self.heads, -1, self.D)[:, :n] for c, s in ((self.k, self.ks), (self.v, self.vs)))


def attention(cache, q, scale, softcap=0.0, slopes=None):
    """(out, allowed error before the output's rounding), float64 [T, q heads, D]."""
    T, Hq, D = q.shape
    group = Hq // cache.heads
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    at = 0
    for b, n in enumerate(cache.new):
        length = cache.lens[b]
        k, v = cache.values(b, length)
        pos = torch.arange(length - n, length)
        keys = torch.arange(length)
        seen = keys <= pos[:, None]
        for h in range(Hq):
            qh, kh, vh = q[at: at + n, h].double(), k[h // group], v[h // group]
            z = qh @ kh.T * scale
            # fp32 sums of D products in any order, the factors and the exponent's own rounding
            size = qh.abs() @ kh.abs().T * abs(scale)
            if softcap:
                z = softcap * torch.tanh(z / softcap)
                size = size + 8 * softcap
            if slopes is not None:
                bias = slopes[h].double() * (keys - pos[:, None])
                z = z + bias
                size = size + bias.abs()
            delta = ((D + 16) * 2.0 ** -24 * size)
            z = torch.where(seen, z, -math.inf)
            p = torch.softmax(z, -1)
            mag = torch.where(seen, p * (2.0 ** -11 + 2.0 ** -18 + 2 * delta), 0)
            out[at: at + n, h] = p @ vh
            tol[at: at + n, h] = mag @ vh.abs() + (p * delta).sum(-1, keepdim=True) * (p @ vh.abs())
            # fp16 below its normal range: 2^-25 of the largest scale's power of two per token,
            # relative to the largest probability
            top = p.max(-1, keepdim=True).values
            tol[at: at + n, h] += top * length * 2.0 ** -25 * 2 * vh.abs().max()
        at += n
    return out, tol
