"""The decoder-block operators that are measured: rotary positions, the append to a paged 8-bit
key/value cache, and the attention over that cache.

Each case names one operator and its sizes.  `run` computes it in a plain form, elementary
torch operations in 32 bits, or, where `own` is true, through this package's entry points.

    rotary   x[t, h, :R] rotated by the angles of position p[t], the rest copied
    append   new keys (rotated) and values quantised to e4m3 with one scale per page and head,
             the page's older tokens re-quantised where its scale grows; queries rotated
    attend   softmax(cap(q k) + distance bias) v over each sequence's cached tokens, causal

The cache: k, v [pages, kv heads, page size, head size] e4m3, scales [pages, kv heads] float32,
page_table [sequences, pages per sequence] int32, lens [sequences] int32 counting the new
tokens, starts [sequences + 1] int32 bounding each sequence's rows among the new tokens.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
SCALE_MIN = 2.0 ** -64


# ------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------

def _rotary(name, T, H, D, R, dtype, layout, inverse=False, pad=0, span=4096):
    """`pad`: heads of the fused projection's row that are not rotated (its values)."""
    return {"name": name, "op": "rotary", "T": T, "H": H, "D": D, "R": R, "dtype": dtype,
            "layout": layout, "inverse": inverse, "pad": pad, "span": span}


def _append(name, B, new, past, Hq, Hkv, D, R, page, dtype, layout, even=False):
    """`new`, `past`: the most new and older tokens of a sequence; `even`: every one has them."""
    return {"name": name, "op": "append", "B": B, "new": new, "past": past, "Hq": Hq, "Hkv": Hkv,
            "D": D, "R": R, "page": page, "dtype": dtype, "layout": layout, "even": even}


def _attend(name, B, new, past, Hq, Hkv, D, page, dtype, cap=0.0, slopes=False, even=False):
    return {"name": name, "op": "attend", "B": B, "new": new, "past": past, "Hq": Hq, "Hkv": Hkv,
            "D": D, "page": page, "dtype": dtype, "cap": cap, "slopes": slopes, "even": even}


def listed():
    return [
        # one decode step of 64 sequences: 32 query and 8 key heads of a fused projection's rows
        _rotary("rotary-step", 64, 40, 128, 128, "bf16", "half", pad=8),
        # a training batch, half of each head rotated in pairs
        _rotary("rotary-train", 16384, 40, 128, 64, "f16", "interleaved", pad=8),
        # the gradient of a training batch: the inverse rotation
        _rotary("rotary-grad", 8193, 12, 64, 64, "bf16", "half", inverse=True),
        # one token of one short sequence in a block of the FFN chain's width (256 = 4 x 64)
        _append("append-one", 1, 1, 200, 4, 4, 64, 64, 16, "bf16", "half", even=True),
        # a decode step of 64 sequences of different lengths
        _append("append-step", 64, 1, 4096, 32, 8, 128, 128, 64, "bf16", "half"),
        # ragged prompts, some of them continuing older pages
        _append("append-prompt", 16, 2048, 1024, 32, 8, 128, 64, 32, "f16", "interleaved"),
        # one token of one short sequence: latency
        _attend("attend-one", 1, 1, 200, 4, 4, 64, 16, "bf16", even=True),
        # a decode step over ragged lengths
        _attend("attend-step", 64, 1, 4096, 32, 8, 128, 64, "bf16"),
        # a full decode batch: the cache's bytes are everything
        _attend("attend-full", 128, 1, 8192, 32, 8, 128, 64, "bf16", even=True),
        # one very long context, work only along the sequence
        _attend("attend-long", 1, 1, 250001, 16, 2, 128, 128, "f16", even=True),
        # drafts of a few tokens checked at once, wide heads, capped scores, distance bias
        _attend("attend-draft", 24, 5, 3000, 16, 8, 256, 32, "bf16", cap=50.0, slopes=True),
        # ragged prompts, chunks over an older context: the products are everything
        _attend("attend-prompt", 4, 2048, 4096, 32, 8, 128, 64, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attend", "attend"])
    dtype = rng.choice(["f16", "bf16"])
    layout = rng.choice(["half", "interleaved"])
    if op == "rotary":
        D = rng.choice([64, 96, 128, 256])
        H = _log(rng, 2, 40)
        T = _log(rng, 1, max(1, min(40000, 80_000_000 // (H * D))))
        c = _rotary("", T, H, D, rng.choice([D, D // 2]), dtype, layout, rng.random() < 0.5,
                    rng.choice([0, 0, 3]), rng.choice([4096, 131072]))
    else:
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        D = rng.choice([64, 64, 128, 128, 96, 256])
        page = rng.choice([16, 32, 64, 128])
        shape = rng.choice(["step", "step", "draft", "prompt"])
        if shape == "prompt":
            B, new, past = rng.randint(1, 4), _log(rng, 32, 1500), _log(rng, 1, 4000)
        else:
            B, new = _log(rng, 1, 128), 1 if shape == "step" else rng.randint(2, 8)
            past = _log(rng, 1, max(2, min(100_000, 200_000_000 // (B * Hkv * D))))
        even = rng.random() < 0.3
        if op == "append":
            c = _append("", B, new, past, Hq, Hkv, D, rng.choice([D, D // 2]), page, dtype, layout,
                        even)
        else:
            c = _attend("", B, new, past, Hq, Hkv, D, page, dtype, rng.choice([0.0, 0.0, 30.0]),
                        rng.random() < 0.25, even)
    del c["name"]
    return c


def _lengths(case):
    """(older, new) token counts of each sequence: a fixed function of the case."""
    B, new, past = case["B"], case["new"], case["past"]
    if case["even"]:
        return [past] * B, [new] * B
    r = random.Random(B * 1_000_003 + new * 10_007 + past)
    older = [r.randint(past // 8, past) for _ in range(B)]
    fresh = [r.randint(max(1, new // 8), new) for _ in range(B)]
    older[-1], fresh[-1] = past, new
    return older, fresh


def work(case):
    if case["op"] == "rotary":
        n = case["T"] * case["H"] * case["D"]
        rot = case["T"] * case["H"] * case["R"]
        return {"bytes": 4 * n + 4 * case["R"] * min(case["T"], case["span"]) + 4 * case["T"],
                "flops": 3 * rot}
    older, fresh = _lengths(case)
    Hq, Hkv, D, T = case["Hq"], case["Hkv"], case["D"], sum(fresh)
    if case["op"] == "append":
        pages = sum((a + n - 1) // case["page"] - a // case["page"] + 1
                    for a, n in zip(older, fresh))
        reads = T * (Hq + 2 * Hkv) * D * 2 + 4 * T * case["R"]
        writes = T * Hq * D * 2 + T * 2 * Hkv * D + 2 * 4 * pages * Hkv
        return {"bytes": reads + writes,
                "flops": T * (3 * (Hq + Hkv) * case["R"] + 4 * Hkv * D)}
    cached = sum(a + n for a, n in zip(older, fresh))
    pairs = sum(n * a + n * (n + 1) // 2 for a, n in zip(older, fresh))
    return {"bytes": cached * Hkv * D * 2 + 8 * Hkv * cached // case["page"] + 4 * T * Hq * D,
            "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------

def _table(span, R):
    """(cos, sin) of position * 10000^(-2 i / R), [span, R / 2, 2] float32."""
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    angle = torch.arange(span, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], -1).float()


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _pool(g, pages, Hkv, page, D):
    """A cache's pages as appends leave them: keys with a few strong channels, values without."""
    scale = torch.exp(0.3 * _randn(g, pages, Hkv)) * (4.0 / F8_MAX)
    gain = torch.ones(D, device="cuda")
    gain[:: max(1, D // 4)] = 4.0
    codes = torch.empty(pages, Hkv, page, D, dtype=F8, device="cuda")
    for at in range(0, pages, 4096):
        n = min(4096, pages - at)
        codes[at: at + n] = (_randn(g, n, Hkv, page, D) * (gain * (F8_MAX / 16))).clamp(
            -F8_MAX, F8_MAX).to(F8)
    return codes, scale


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "rotary":
        T, H, D = case["T"], case["H"], case["D"]
        rows = _randn(g, T, H + case["pad"], D).to(dt)
        s["x"] = rows[:, :H]
        s["table"] = _table(case["span"], case["R"])
        s["positions"] = torch.randint(case["span"], (T,), generator=g, device="cuda",
                                       dtype=torch.int32)
        return s
    B, Hq, Hkv, D, page = (case[k] for k in ("B", "Hq", "Hkv", "D", "page"))
    older, fresh = _lengths(case)
    lens = [a + n for a, n in zip(older, fresh)]
    need = [-(-n // page) for n in lens]
    pages, T = sum(need) + 5, sum(fresh)
    s["k_cache"], s["k_scale"] = _pool(g, pages, Hkv, page, D)
    s["v_cache"], s["v_scale"] = _pool(g, pages, Hkv, page, D)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    slot = torch.arange(max(need), device="cuda")
    first = torch.tensor(_starts(need)[:-1], device="cuda")
    used = slot < torch.tensor(need, device="cuda")[:, None]
    s["page_table"] = torch.where(used, order[(first[:, None] + slot).clamp_max(pages - 1)], -1)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["starts"] = torch.tensor(_starts(fresh), dtype=torch.int32, device="cuda")
    s["max_new"] = max(fresh)
    rows = _randn(g, T, Hq + 2 * Hkv, D).to(dt)      # the fused projection of the new tokens
    s["q"], s["k"], s["v"] = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    if case["op"] == "append":
        s["table"] = _table(max(lens), case["R"])
    else:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq).float() \
            if case["slopes"] else None
    return s


# ------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------

def _rotate(x, cos_sin, layout, inverse=False):
    """x [T, H, D] float32 rotated by cos_sin [T, R / 2, 2]; channels past R are copied."""
    half = cos_sin.shape[1]
    cos, sin = cos_sin[:, None, :, 0], cos_sin[:, None, :, 1]
    if inverse:
        sin = -sin
    if layout == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _tokens(s, T):
    """Of each new token: its sequence, its place among that sequence's new ones, its position."""
    at = torch.arange(T, device="cuda")
    seq = torch.searchsorted(s["starts"][1:], at.to(torch.int32), right=True)
    starts = s["starts"].long()
    i = at - starts[seq]
    count = starts[1:] - starts[:-1]
    return seq, i, (s["lens"] - count)[seq] + i


def _append_pool(s, new, codes, scale, seq, pos):
    """Writes new [T, Hkv, D] float32 into one pool (codes and scales)."""
    page = codes.shape[2]
    table = s["page_table"].long()
    count = s["starts"][1:] - s["starts"][:-1]
    start = (s["lens"] - count).long()
    where = table[seq, pos // page]
    size = torch.where(new.isfinite(), new.abs(), 0).amax(-1)
    most = torch.zeros_like(scale).index_reduce_(0, where, size, "amax")
    begun = (pos // page * page < start[seq])[:, None]           # the page holds older tokens
    before = torch.where(begun, scale[where], 0)
    after = torch.maximum(before, most[where] / F8_MAX).clamp_min(SCALE_MIN)
    # the older tokens of each sequence's first page, under the new scale
    first = table.gather(1, (start // page)[:, None])[:, 0]
    head = s["starts"][:-1].long()
    old = codes[first].float()
    ratio = torch.where(begun[head], before[head] / after[head], 1)
    held = torch.arange(page, device="cuda") < (start % page)[:, None]
    codes[first] = torch.where(held[:, None, :, None], (old * ratio[:, :, None, None]), old).to(F8)
    codes[where, :, pos % page] = (new / after[:, :, None]).clamp(-F8_MAX, F8_MAX).to(F8)
    scale[where] = after


def _run_plain(s):
    case = s["case"]
    if case["op"] == "rotary":
        turned = _rotate(s["x"].float(), s["table"][s["positions"].long()], case["layout"],
                         case["inverse"])
        return turned.to(s["x"].dtype)
    q = s["q"]
    T, Hq, D = q.shape
    seq, i, pos = _tokens(s, T)
    if case["op"] == "append":
        angles = s["table"][pos]
        k = _rotate(s["k"].float(), angles, case["layout"])
        _append_pool(s, k, s["k_cache"], s["k_scale"], seq, pos)
        _append_pool(s, s["v"].float(), s["v_cache"], s["v_scale"], seq, pos)
        turned = _rotate(q.float(), angles, case["layout"]).to(q.dtype)
        return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"],
                "v_scale": s["v_scale"], "q": turned}
    B, Hkv, page, n = case["B"], case["Hkv"], case["page"], s["max_new"]
    table = s["page_table"].long().clamp_min(0)
    k, v = ((s[c][table].float() * s[z][table][..., None, None]).transpose(1, 2).reshape(
        B, Hkv, -1, D) for c, z in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
    keys = torch.arange(k.shape[2], device="cuda")
    v = v.masked_fill((keys >= s["lens"][:, None])[:, None, :, None], 0)
    rows = torch.zeros(B, n, Hq, D, device="cuda")
    rows[seq, i] = q.float()
    at = torch.zeros(B, n, dtype=torch.long, device="cuda")
    at[seq, i] = pos
    rows = rows.reshape(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = (rows @ k.transpose(2, 3)).reshape(B, Hq, n, -1) * D ** -0.5
    if case["cap"]:
        score = torch.tanh(score / case["cap"]) * case["cap"]
    if case["slopes"]:
        score = score + s["slopes"][:, None, None] * (keys - at[:, None, :, None])
    score = score.masked_fill((keys > at[..., None])[:, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).reshape(B, Hkv, -1, k.shape[2])
    out = (p @ v).reshape(B, Hkv, Hq // Hkv, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    return out[seq, i].to(q.dtype)


def _run_own(s):
    from gemm_conv_chains_gb300 import ops
    case = s["case"]
    if case["op"] == "rotary":
        return ops.rotary(s["x"], s["table"], s["positions"], case["layout"], case["inverse"])
    if case["op"] == "append":
        q = ops.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                             s["page_table"], s["lens"], s["starts"], s["max_new"],
                             table=s["table"], layout=case["layout"], q=s["q"])
        return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"],
                "v_scale": s["v_scale"], "q": q}
    return ops.cache_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                               s["page_table"], s["lens"], s["starts"], s["max_new"],
                               softcap=case["cap"], slopes=s["slopes"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------

def _turn(x, position, case, table, sign=1.0):
    """x [T, H, D] float64: each pair (a, b) becomes (a + i b) e^(i angle)."""
    R = case["R"]
    cs = table[position].double()
    z = torch.complex(cs[..., 0], sign * cs[..., 1])[:, None]
    y = x.clone()
    first = slice(0, R // 2) if case["layout"] == "half" else slice(0, R, 2)
    second = slice(R // 2, R) if case["layout"] == "half" else slice(1, R, 2)
    w = torch.complex(x[..., first], x[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _exact_append(s, case):
    older, fresh = _lengths(case)
    page = case["page"]
    table = s["page_table"].tolist()
    out = {"k": s["k_cache"].double(), "v": s["v_cache"].double(),
           "k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double(),
           "q": torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")}
    at = 0
    for b, (a, n) in enumerate(zip(older, fresh)):
        position = torch.arange(a, a + n, device="cuda")
        out["q"][at: at + n] = _turn(s["q"][at: at + n].double(), position, case, s["table"])
        news = {"k": _turn(s["k"][at: at + n].double(), position, case, s["table"]),
                "v": s["v"][at: at + n].double()}
        for name, x in news.items():
            codes, scale = out[name], out[name + "_scale"]
            for j in range(a // page, (a + n - 1) // page + 1):
                lo, hi = max(a, j * page), min(a + n, (j + 1) * page)
                part = x[lo - a: hi - a].transpose(0, 1)             # [Hkv, tokens, D]
                at_page = table[b][j]
                held = max(0, a - j * page)
                was = scale[at_page].clone() if held else torch.zeros_like(scale[at_page])
                now = torch.maximum(was, part.abs().amax((1, 2)) / F8_MAX).clamp_min(SCALE_MIN)
                keep = codes[at_page][:, :held] * (was / now)[:, None, None]
                codes[at_page][:, :held] = keep.to(F8).double()
                codes[at_page][:, lo - j * page: hi - j * page] = \
                    (part / now[:, None, None]).to(F8).double()
                scale[at_page] = now
        at += n
    return out


def _exact_attend(s, case):
    older, fresh = _lengths(case)
    Hq, Hkv, D, page = (case[k] for k in ("Hq", "Hkv", "D", "page"))
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (a, n) in enumerate(zip(older, fresh)):
        pages = s["page_table"][b, : -(-(a + n) // page)].long()
        keys = torch.arange(a + n, device="cuda")
        position = torch.arange(a, a + n, device="cuda")[:, None]
        for h in range(Hkv):
            k, v = ((s[c][pages, h].double() * s[z][pages, h].double()[:, None, None]).reshape(
                -1, D)[: a + n] for c, z in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
            for j in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                z = s["q"][at: at + n, j].double() @ k.T / math.sqrt(D)
                if case["cap"]:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                if case["slopes"]:
                    z = z + s["slopes"][j].double() * (keys - position)
                z = torch.where(keys <= position, z, -math.inf)
                out[at: at + n, j] = torch.softmax(z, -1) @ v
        at += n
    return out


def exact(case, seed):
    if case["op"] == "attend" and work(case)["flops"] > 2.5e12:
        return None                                  # over 20 seconds in 64 bits
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _turn(s["x"].double(), s["positions"].long(), case, s["table"],
                     -1.0 if case["inverse"] else 1.0)
    return _exact_append(s, case) if case["op"] == "append" else _exact_attend(s, case)
