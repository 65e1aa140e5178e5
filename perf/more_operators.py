"""The operators of drafted and branching sequences that are measured: attention for trees of drafted
tokens over the paged 8-bit key/value cache, and what happens to the cache's pages when sequences
branch, end, grow or keep only some of their tokens.

Each case names one operator and its sizes.  `run` computes it in a plain form, elementary torch
operations in 32 bits, or, where `own` is true, through this package's entry points.

    tree     softmax(cap(q k) + distance bias) v of drafted tokens over their sequence's older tokens
             and, of the drafted ones, those that a row's mask names (its ancestors in the tree)
    compact  the kept tokens of each sequence moved together, a page's codes re-quantised where tokens
             of a page with a larger scale come in
    copy     pages copied to others, each up to a count of tokens
    pages    the page table after sequences branch (beams), end, lose their last tokens and make room
             for new ones: pages shared by several sequences, a page that one of them writes
             on copied first, free pages found by what the table does not name

The cache: k, v [pages, kv heads, page size, head size] e4m3, scales [pages, kv heads] float32,
page_table [sequences, pages per sequence] int32, lens [sequences] int32.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
SINKS = 4           # first tokens that an eviction always keeps


# ------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------

def _tree(name, B, new, past, Hq, Hkv, D, page, dtype, cap=0.0, slopes=False, even=False):
    """`new`, `past`: the most drafted and older tokens of a sequence; `even`: every one has them."""
    return {"name": name, "op": "tree", "B": B, "new": new, "past": past, "Hq": Hq, "Hkv": Hkv,
            "D": D, "page": page, "dtype": dtype, "cap": cap, "slopes": slopes, "even": even}


def _compact(name, B, span, past, keep, Hkv, D, page, even=False):
    """Of the `span` tokens behind `past` older ones `keep` stay, at most each."""
    return {"name": name, "op": "compact", "B": B, "new": span, "past": past, "keep": keep,
            "Hkv": Hkv, "D": D, "page": page, "even": even}


def _copy(name, N, Hkv, D, page, whole=False):
    """`whole`: every page is copied to its end."""
    return {"name": name, "op": "copy", "N": N, "Hkv": Hkv, "D": D, "page": page, "whole": whole}


def _pages(name, B, rows, past, new, page, spare, shared):
    """`rows` sequences follow on B; `shared`: the share of them that branch off another's."""
    return {"name": name, "op": "pages", "B": B, "rows": rows, "past": past, "new": new,
            "page": page, "spare": spare, "shared": shared}


def listed():
    return [
        # eight drafted tokens of one short sequence: latency
        _tree("tree-one", 1, 8, 200, 4, 4, 64, 16, "bf16", even=True),
        # small trees of a batch of sequences of different lengths
        _tree("tree-step", 32, 8, 4096, 32, 8, 128, 64, "bf16"),
        # wide trees: the products count beside the cache's bytes
        _tree("tree-wide", 16, 60, 4096, 32, 8, 128, 64, "bf16"),
        # a wide tree on one very long context, work only along the sequence
        _tree("tree-long", 1, 64, 131072, 16, 2, 128, 128, "f16", even=True),
        # trees with wide heads, capped scores, distance bias
        _tree("tree-bias", 24, 13, 3000, 16, 8, 256, 32, "bf16", cap=50.0, slopes=True),
        # the accepted path of each sequence's drafts moved together: a few tokens each
        _compact("compact-accept", 64, 16, 4096, 6, 8, 128, 64),
        # half of a full batch's tokens evicted: the bytes are everything
        _compact("compact-evict", 16, 8192 - SINKS, SINKS, 4096, 8, 128, 64, even=True),
        # one long sequence of few heads thinned out
        _compact("compact-long", 1, 100001, SINKS, 30011, 2, 64, 128, even=True),
        # two beams of a short sequence part: latency
        _copy("copy-two", 2, 2, 64, 16),
        # whole prompts copied: the bytes are everything
        _copy("copy-prompts", 1536, 8, 128, 64, whole=True),
        # a step of 64 beams, some of which branch
        _pages("pages-beams", 64, 64, 1500, 1, 16, 200, 0.25),
        # a large serving batch: sequences end, others branch off a shared prompt and grow
        _pages("pages-serve", 512, 480, 8000, 300, 32, 30000, 0.125),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "compact", "copy", "pages"])
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 64, 128, 128, 96, 256])
    page = rng.choice([16, 32, 64, 128])
    even = rng.random() < 0.3
    if op == "tree":
        new = _log(rng, 1, 150)
        B = _log(rng, 1, max(2, min(64, 1000 // new)))
        past = _log(rng, 1, max(2, min(60_000, 60_000_000 // (B * Hkv * D),
                                       2_500_000_000 // (B * new * Hkv * D))))
        c = _tree("", B, new, past, Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv, D, page,
                  rng.choice(["f16", "bf16"]), rng.choice([0.0, 0.0, 30.0]), rng.random() < 0.25,
                  even)
    elif op == "compact":
        B = _log(rng, 1, 64)
        if rng.random() < 0.5:                       # an accepted path
            span, past = rng.randint(2, 64), _log(rng, 1, max(2, 30_000_000 // (B * Hkv * D)))
            keep = rng.randint(1, min(span, 9))
        else:                                        # an eviction
            span = _log(rng, 20, max(40, min(60_000, 60_000_000 // (B * Hkv * D))))
            past, keep = rng.choice([0, SINKS]), _log(rng, 10, span)
        c = _compact("", B, span, past, keep, Hkv, D, page, even)
    elif op == "copy":
        c = _copy("", _log(rng, 1, max(2, min(2000, 90_000_000 // (Hkv * D * page)))), Hkv, D, page,
                  even)
    else:
        B = _log(rng, 1, 400)
        rows = max(1, min(512, round(B * rng.uniform(0.5, 1.5))))
        c = _pages("", B, rows, _log(rng, 1, 12_000_000 // B // 16), _log(rng, 1, 300), page,
                   rng.choice([0, 100, 5000]) + rows * 40, rng.choice([0.0, 0.25, 1.0]))
    del c["name"]
    return c


def _random(case):
    return random.Random(case["B"] * 1_000_003 + case["new"] * 10_007 + case["past"])


def _lengths(case):
    """(older, further) token counts of each sequence: a fixed function of the case."""
    B, new, past = case["B"], case["new"], case["past"]
    if case["even"]:
        return [past] * B, [new] * B
    r = _random(case)
    older = [r.randint(past // 8, past) for _ in range(B)]
    fresh = [r.randint(max(1, new // 8), new) for _ in range(B)]
    older[-1], fresh[-1] = past, new
    return older, fresh


def _counts(case):
    """Of each sequence of a compaction, how many of its further tokens stay."""
    fresh = _lengths(case)[1]
    if case["even"]:
        return [case["keep"]] * case["B"]
    r = _random(case)
    return [min(n, r.randint(0, case["keep"])) for n in fresh[:-1]] + [case["keep"]]


def _copied(case):
    """Tokens of each copied page."""
    r = random.Random(case["N"] * 1_009 + case["page"])
    return [case["page"] if case["whole"] else r.randint(1, case["page"])
            for _ in range(case["N"])]


def _branches(case):
    """(lens of the B sequences, parents, kept tokens and new tokens of the rows that follow)."""
    r = random.Random(case["B"] * 1_000_003 + case["rows"] * 10_007 + case["past"])
    B, rows, past = case["B"], case["rows"], case["past"]
    lens = [r.randint(past // 8, past) for _ in range(B)]
    parents, kept, new = [], [], []
    for i in range(rows):
        x = r.random()
        p = i if i < B else -1                       # goes on, or is a new sequence
        if x < case["shared"]:
            p = r.randrange(B)                       # branches off
        parents.append(p)
        have = lens[p] if p >= 0 else 0
        cut = r.random()                             # some lose their last tokens or branch earlier
        kept.append(have if cut < 0.75 else max(0, have - r.randint(0, 40)) if cut < 0.95 else
                    have // 2)
        new.append(0 if r.random() < 0.05 else r.randint(max(1, case["new"] // 8), case["new"]))
    return lens, parents, kept, new


def work(case):
    if case["op"] == "tree":
        older, fresh = _lengths(case)
        Hq, Hkv, D, T = case["Hq"], case["Hkv"], case["D"], sum(fresh)
        cached = sum(a + n for a, n in zip(older, fresh))
        pairs = sum(n * (a + 1) for a, n in zip(older, fresh))     # older tokens, and a row's own
        return {"bytes": cached * Hkv * D * 2 + 8 * Hkv * cached // case["page"] + 4 * T * Hq * D +
                8 * T * -(-case["new"] // 64), "flops": 4 * pairs * Hq * D}
    if case["op"] == "compact":
        moved = sum(_counts(case))
        n = moved * case["Hkv"] * case["D"] * 2
        return {"bytes": 2 * n + 4 * moved, "flops": 2 * n}
    if case["op"] == "copy":
        return {"bytes": 4 * sum(_copied(case)) * case["Hkv"] * case["D"] + 12 * case["N"],
                "flops": 0}
    kept = _branches(case)[2]
    page = case["page"]
    read = sum(-(-a // page) for a in kept) + 4 * case["rows"]
    return {"bytes": 4 * (read + case["rows"] * (_width(case) + 4)), "flops": read}


# ------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


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


def _pools(g, s, pages, Hkv, page, D):
    s["k_cache"], s["k_scale"] = _pool(g, pages, Hkv, page, D)
    s["v_cache"], s["v_scale"] = _pool(g, pages, Hkv, page, D)


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _page_lists(g, need, pages, width):
    """A page table whose rows have need[b] pages in any order of the pool, -1 behind them."""
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    slot = torch.arange(width, device="cuda")
    first = torch.tensor(_starts(need)[:-1], device="cuda")
    used = slot < torch.tensor(need, device="cuda")[:, None]
    return torch.where(used, order[(first[:, None] + slot).clamp_max(pages - 1)], -1)


def _width(case):
    """Pages per row of the table of a `pages` case."""
    return -(-(case["past"] + case["new"]) // case["page"])


def _masks(seed, fresh, words):
    """Random trees: (masks [T, words] int64, depth [T]) of each node's ancestors and itself."""
    r = random.Random(seed)
    masks, depth = [], []
    for n in fresh:
        seen, deep = [], []
        for i in range(n):
            parent = r.randint(max(0, i - 1 - i // 3), i - 1) if i else -1
            seen.append((seen[parent] if i else 0) | 1 << i)
            deep.append(deep[parent] + 1 if i else 0)
        for m in seen:
            masks.append([(m >> 64 * w & (1 << 64) - 1) - (m >> 64 * w + 63 & 1) * (1 << 64)
                          for w in range(words)])
        depth += deep
    return torch.tensor(masks, dtype=torch.int64, device="cuda"), _ints(depth)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "pages":
        lens, parents, kept, new = _branches(case)
        page, width = case["page"], _width(case)
        need = [-(-n // page) for n in lens]
        s["pages"] = sum(need) + case["spare"]
        s["page_table"] = _page_lists(g, need, s["pages"], width)
        s["lens"], s["parents"], s["kept"], s["new"] = map(_ints, (lens, parents, kept, new))
        # the tables of a program that keeps two and takes them in turn
        s["out"] = (torch.empty(len(parents), width, dtype=torch.int32, device="cuda"),
                    torch.empty(len(parents), dtype=torch.int32, device="cuda"),
                    torch.empty(len(parents), 3, dtype=torch.int32, device="cuda"),
                    torch.empty(1, dtype=torch.int32, device="cuda"))
        return s
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    if case["op"] == "copy":
        N = case["N"]
        _pools(g, s, 2 * N + 3, Hkv, page, D)
        order = torch.randperm(2 * N + 3, generator=g, device="cuda").to(torch.int32)
        s["copies"] = torch.stack([order[:N], order[N: 2 * N], _ints(_copied(case))], 1)
        return s
    older, fresh = _lengths(case)
    lens = [a + n for a, n in zip(older, fresh)]
    need = [-(-n // page) for n in lens]
    pages, T = sum(need) + 5, sum(fresh)
    _pools(g, s, pages, Hkv, page, D)
    s["page_table"] = _page_lists(g, need, pages, max(need))
    s["lens"] = _ints(lens)
    if case["op"] == "compact":
        counts = _counts(case)
        s["first"], s["counts"] = _ints(older), _ints(counts)
        # the kept tokens: the least of random numbers, in order
        at = torch.arange(case["new"], device="cuda")
        x = torch.rand(case["B"], case["new"], generator=g, device="cuda")
        x.masked_fill_(at >= _ints(fresh)[:, None], 2.0)
        stays = x.argsort(-1).argsort(-1) < s["counts"][:, None]
        gone = torch.iinfo(torch.int32).max
        kept = torch.where(stays, s["first"][:, None] + at, gone).sort(-1).values[:, :max(counts)]
        s["tokens"] = torch.where(kept == gone, -1, kept).to(torch.int32).contiguous()
        return s
    Hq = case["Hq"]
    s["starts"] = _ints(_starts(fresh))
    s["max_new"] = max(fresh)
    s["masks"], depth = _masks(seed, fresh, -(-s["max_new"] // 64))
    s["positions"] = depth + torch.repeat_interleave(_ints(older), _ints(fresh).long())
    rows = _randn(g, T, Hq + 2 * Hkv, D).to(DTYPES[case["dtype"]])
    s["q"] = rows[:, :Hq]                            # of the fused projection of the new tokens
    s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq).float() \
        if case["slopes"] else None
    return s


# ------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------

def _plain_tree(s, case):
    q, table = s["q"], s["page_table"].long().clamp_min(0)
    T, Hq, D = q.shape
    B, Hkv, n = case["B"], case["Hkv"], s["max_new"]
    k, v = ((s[c][table].float() * s[z][table][..., None, None]).transpose(1, 2).reshape(
        B, Hkv, -1, D) for c, z in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
    L = k.shape[2]
    keys = torch.arange(L, device="cuda")
    v = v.masked_fill((keys >= s["lens"][:, None])[:, None, :, None], 0)
    # of each new token: its sequence, its place among that sequence's new ones
    at = torch.arange(T, device="cuda")
    seq = torch.searchsorted(s["starts"][1:], at.to(torch.int32), right=True)
    starts = s["starts"].long()
    i = at - starts[seq]
    first = s["lens"].long() - (starts[1:] - starts[:-1])
    # which tokens each row sees: the older ones, and the new ones of its mask
    local = keys - first[:, None]                                                   # [B, L]
    inside = (local >= 0) & (keys < s["lens"][:, None])
    bit = torch.where(inside, local, 0)
    word = s["masks"].gather(1, (bit // 64)[seq])
    sees = (local < 0)[seq] | (inside[seq] & ((word >> (bit % 64)[seq]) & 1).bool())
    seen = torch.zeros(B, n, L, dtype=torch.bool, device="cuda")
    seen[seq, i] = sees
    rows = torch.zeros(B, n, Hq, D, device="cuda")
    rows[seq, i] = q.float()
    rows = rows.reshape(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = (rows @ k.transpose(2, 3)).reshape(B, Hq, n, L) * D ** -0.5
    if case["cap"]:
        score = torch.tanh(score / case["cap"]) * case["cap"]
    if case["slopes"]:
        place = torch.zeros(B, n, dtype=torch.long, device="cuda")
        place[seq, i] = s["positions"].long()
        key_at = torch.where(inside, s["positions"].long()[(starts[:-1, None] + bit).clamp_max(T - 1)],
                             keys)
        score = score + s["slopes"][:, None, None] * (key_at[:, None] - place[..., None])[:, None]
    score = score.masked_fill(~seen[:, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp_min(-1e30))
    p = (p / p.sum(-1, keepdim=True).clamp_min(1e-30)).reshape(B, Hkv, -1, L)
    out = (p @ v).reshape(B, Hkv, Hq // Hkv, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    return out[seq, i].to(q.dtype)


def _plain_compact(s, case):
    page = case["page"]
    table, tokens = s["page_table"].long(), s["tokens"].long()
    seq, i = (torch.arange(tokens.shape[1], device="cuda") < s["counts"][:, None]).nonzero(
        as_tuple=True)
    first = s["first"].long()
    come, go = tokens[seq, i], first[seq] + i
    from_page, to_page = table[seq, come // page], table[seq, go // page]
    # the pages that older tokens share with moved ones
    b = ((first % page != 0) & (s["counts"] > 0)).nonzero()[:, 0]
    head = table[b, first[b] // page]
    held = torch.arange(page, device="cuda") < (first[b] % page)[:, None]
    for codes, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        had = scale[from_page]
        most = torch.zeros_like(scale).index_reduce_(0, to_page, had, "amax")
        most.index_reduce_(0, head, scale[head], "amax")
        moved = codes[from_page, :, come % page].float()
        old = codes[head].float()
        old_ratio = torch.where(scale[head] == most[head], 1, scale[head] / most[head])
        codes[head] = torch.where(held[:, None, :, None], old * old_ratio[:, :, None, None],
                                  old).to(F8)
        ratio = torch.where(had == most[to_page], 1, had / most[to_page])
        codes[to_page, :, go % page] = (moved * ratio[:, :, None]).to(F8)
        scale[to_page] = most[to_page]
    return {c: s[c] for c in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _plain_copy(s, case):
    come, go, count = s["copies"].long().unbind(1)
    taken = torch.arange(case["page"], device="cuda") < count[:, None]
    for codes, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        raw = codes.view(torch.uint8)
        raw[go] = torch.where(taken[:, None, :, None], raw[come], raw[go])
        scale[go] = scale[come]
    return {c: s[c] for c in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _plain_pages(s, case):
    page, pages, parents = case["page"], s["pages"], s["parents"].long()
    rows, width = parents.shape[0], s["page_table"].shape[1]
    kept, total = s["kept"].long(), s["kept"].long() + s["new"].long()
    table = s["page_table"].long()[parents.clamp_min(0)]
    slot = torch.arange(width, device="cuda")
    row = torch.arange(rows, device="cuda")
    have = (kept + page - 1) // page
    # who holds each page: 0 a row that only reads it, r + 1 the lowest row that writes on its end
    writes = (kept % page != 0) & (total > kept)
    writing = writes[:, None] & (slot == (kept // page)[:, None])
    holds = slot < have[:, None]
    nobody = rows + 1
    owner = torch.full((pages,), nobody, device="cuda").scatter_reduce_(
        0, table[holds], torch.where(writing, row[:, None] + 1, 0)[holds], "amin")
    last = table.gather(1, (kept // page).clamp_max(width - 1)[:, None])[:, 0]
    copy = writes & (owner[last.clamp_min(0)] != row + 1)
    begin = have - copy.long()
    need = (total + page - 1) // page - begin
    rank = need.cumsum(0) - need
    free = (owner == nobody).nonzero()[:, 0]
    n_free = free.shape[0]
    free = torch.cat([free, torch.full((1,), -1, device="cuda")])
    fresh = (slot >= begin[:, None]) & (slot < ((total + page - 1) // page)[:, None])
    given = free[(rank[:, None] + slot - begin[:, None]).clamp(0, n_free)]
    out = torch.where(fresh, given, torch.where(holds, table, -1))
    to = free[rank.clamp_max(n_free)]
    done = copy & (to >= 0)
    copies = torch.stack([torch.where(done, last, -1), torch.where(done, to, -1),
                          torch.where(done, kept % page, 0)], 1)
    left = n_free - need.sum()
    return tuple(x.to(torch.int32) for x in (out, total, copies, left.reshape(1)))


def _run_plain(s):
    case = s["case"]
    return {"tree": _plain_tree, "compact": _plain_compact, "copy": _plain_copy,
            "pages": _plain_pages}[case["op"]](s, case)


def _run_own(s):
    from gemm_conv_chains_gb300 import ops
    case = s["case"]
    if case["op"] == "pages":
        return ops.cache_pages(s["page_table"], s["lens"], s["pages"], case["page"], s["parents"],
                               s["kept"], s["new"], out=s["out"])
    cache = [s[c] for c in ("k_cache", "v_cache", "k_scale", "v_scale")]
    if case["op"] == "tree":
        return ops.cache_tree_attention(s["q"], s["masks"], *cache, s["page_table"], s["lens"],
                                        s["starts"], s["max_new"], positions=s["positions"],
                                        softcap=case["cap"], slopes=s["slopes"])
    if case["op"] == "compact":
        ops.cache_compact(*cache, s["page_table"], s["lens"], s["first"], s["tokens"], s["counts"])
    else:
        ops.cache_copy(*cache, s["copies"])
    return dict(zip(("k_cache", "v_cache", "k_scale", "v_scale"), cache))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------

def _exact_tree(s, case):
    older, fresh = _lengths(case)
    Hq, Hkv, D, page = (case[k] for k in ("Hq", "Hkv", "D", "page"))
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    bits = torch.arange(64, device="cuda")
    row = 0
    for b, (a, n) in enumerate(zip(older, fresh)):
        mine = slice(row, row + n)
        ids = s["page_table"][b, : -(-(a + n) // page)].long()
        tree = (s["masks"][mine, :, None] >> bits & 1).flatten(1)[:, :n].bool()
        seen = torch.cat([torch.ones(n, a, dtype=torch.bool, device="cuda"), tree], 1)
        where = torch.cat([torch.arange(a, device="cuda"), s["positions"][mine]]).double()
        far = where - s["positions"][mine, None].double()
        for h in range(Hkv):
            k, v = ((s[c][ids, h].double() * s[z][ids, h].double()[:, None, None]).reshape(
                -1, D)[: a + n] for c, z in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
            for j in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                z = s["q"][mine, j].double() @ k.T / math.sqrt(D)
                if case["cap"]:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                if case["slopes"]:
                    z = z + s["slopes"][j].double() * far
                out[mine, j] = torch.softmax(z.masked_fill(~seen, -math.inf), -1) @ v
        row += n
    return out


def _exact_compact(s, case):
    page = case["page"]
    table, firsts, counts = (s[c].tolist() for c in ("page_table", "first", "counts"))
    out = {}
    for pool in ("k", "v"):
        codes, scale = s[pool + "_cache"].double(), s[pool + "_scale"].double()
        for b, (first, n) in enumerate(zip(firsts, counts)):
            ids = torch.tensor(table[b], device="cuda")
            come = torch.cat([torch.arange(first // page * page, first, device="cuda"),
                              s["tokens"][b, :n].long()])
            if n == 0:
                continue
            had = scale[ids[come // page]]                           # [tokens, Hkv]
            value = codes[ids[come // page], :, come % page]
            for j in range(0, come.shape[0], page):
                at = ids[first // page + j // page]
                now = had[j: j + page].amax(0)
                ratio = torch.where(had[j: j + page] == now, 1, had[j: j + page] / now)
                held = value[j: j + page] * ratio[..., None]
                codes[at, :, : held.shape[0]] = held.to(F8).double().transpose(0, 1)
                scale[at] = now
        out[pool + "_cache"], out[pool + "_scale"] = codes, scale
    return out


def _exact_copy(s):
    out = {c: s[c].double() for c in ("k_cache", "v_cache", "k_scale", "v_scale")}
    for come, go, n in s["copies"].tolist():
        for pool in ("k", "v"):
            out[pool + "_cache"][go, :, :n] = out[pool + "_cache"][come, :, :n]
            out[pool + "_scale"][go] = out[pool + "_scale"][come]
    return out


def exact(case, seed):
    if case["op"] == "pages" or case["op"] == "tree" and work(case)["flops"] > 2.5e12:
        return None                                  # whole numbers; over 20 seconds in 64 bits
    s = prepare(case, seed)
    return _exact_copy(s) if case["op"] == "copy" else \
        {"tree": _exact_tree, "compact": _exact_compact}[case["op"]](s, case)
