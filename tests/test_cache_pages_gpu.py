"""What happens to the pages of the e4m3 cache: the page table of a step's sequences, copies of pages
and kept tokens moved together.  Whole numbers and codes have one right answer."""
import random

import pytest
import torch

from gemm_conv_chains_gb300 import ops

import branch_ref as br
import decoder_ref as ref
from decoder_ref import F8

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ops.lib()
    ops.get_cache_error()
    yield
    st, info = ops.get_cache_error()
    assert st == 0, f"cache error word left set: {st} {info}"


def _ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------
# the page table
# ------------------------------------------------------------------------------------

def _table(lens, page, width, pages, seed, shared=0):
    """Rows of random pages; the first `shared` pages of all rows are the same ones."""
    order = list(range(pages))
    random.Random(seed).shuffle(order)
    common = [order.pop() for _ in range(shared)]
    table = []
    for n in lens:
        need = -(-n // page)
        row = common[:need]
        row += [order.pop() for _ in range(need - len(row))]
        table.append(row + [-1] * (width - len(row)))
    return table


def _check_pages(table, lens, pages, page, width, parents=None, kept=None, new=None, **kw):
    want = br.pages(table, lens, pages, page, parents, kept, new)
    got = ops.cache_pages(_ints(table).reshape(len(table), width), _ints(lens).reshape(-1), pages, page,
                          _ints(parents), _ints(kept), _ints(new), **kw)
    for name, g, w in zip(("table", "lens", "copies", "left"), got, want):
        w = torch.tensor(w, dtype=torch.int32).reshape(g.shape)
        assert torch.equal(g.cpu(), w), (name, (g.cpu() != w).nonzero()[:4].tolist(), g.cpu(), w)
    return got


def _random_step(seed, B, rows, page, most, shared=0, new=5, branch=0.4):
    r = random.Random(seed)
    lens = [r.randint(shared * page, most) for _ in range(B)]
    width = -(-(most + new) // page) + r.randint(0, 3)
    parents = [r.randrange(B) if B and r.random() < branch else i if i < B else -1 for i in range(rows)]
    kept = []
    for p in parents:
        n = lens[p] if p >= 0 else 0
        kept.append(r.choice([n, n, n, r.randint(0, n), n // page * page, 0]))
    fresh = [r.choice([0, 1, 1, r.randint(1, new)]) for _ in range(rows)]
    return lens, width, parents, kept, fresh


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("B,rows,page,most,shared", [(1, 1, 16, 40, 0), (3, 5, 16, 100, 2), (8, 8, 64, 500, 0),
                                                     (20, 13, 32, 300, 4), (40, 90, 256, 3000, 1),
                                                     (300, 350, 16, 900, 3)])
def test_steps(seed, B, rows, page, most, shared):
    lens, width, parents, kept, new = _random_step(seed, B, rows, page, most, shared, new=3 * page // 2)
    pages = sum(-(-n // page) for n in lens) + 40 + 3 * rows
    table = _table(lens, page, width, pages, seed, shared)
    _check_pages(table, lens, pages, page, width, parents, kept, new)


def test_large_pools_and_wide_tables():
    """One block on a small pool; three kernels and a workspace on larger ones or for many rows."""
    for pages, B, rows in ((40960, 60, 128), (40961, 60, 70), (1000003, 30, 1500), (45000, 200, 4096),
                           (9000, 40, 129), (327680, 128, 128)):
        lens, width, parents, kept, new = _random_step(pages, B, rows, 16, 4000, 5, new=40)
        table = _table(lens, 16, width, pages, 1, 5)
        got = _check_pages(table, lens, pages, 16, width, parents, kept, new)
        n = -(-pages // 4) * 16 + 16 * rows if pages > 40960 or rows > 128 else 0
        if n:                                        # a workspace of the program's own, whatever it holds
            work = torch.full((n,), 0x11, dtype=torch.uint8, device="cuda")
            again = ops.cache_pages(_ints(table), _ints(lens), pages, 16, _ints(parents), _ints(kept),
                                    _ints(new), workspace=work)
            assert all(torch.equal(a, b) for a, b in zip(got, again))
            with pytest.raises(ops.B2BError, match="SHAPE"):
                ops.cache_pages(_ints(table), _ints(lens), pages, 16, _ints(parents), workspace=work[:64])


def test_defaults():
    lens, page, width = [30, 16, 0, 47], 16, 4
    table = _table(lens, page, width, 20, 0)
    same = _check_pages(table, lens, 20, page, width)
    assert torch.equal(same[0].cpu(), torch.tensor(table, dtype=torch.int32))
    _check_pages(table, lens, 20, page, width, new=[1, 1, 1, 1])
    _check_pages(table, lens, 20, page, width, kept=[3, 16, 0, 32])
    _check_pages(table, lens, 20, page, width, parents=[0, 0, 0, 3, -1, 1])
    _check_pages(table, lens, 20, page, width, parents=[])                  # all end


def test_beams_of_one_sequence_share_and_part():
    """Four beams off a prompt of 20 tokens, page 16: the full page is shared, the first beam goes
    on in the other, three copy it; a fifth that gets no new token makes all four copy."""
    table = [[7, 3, -1, -1]]
    got = _check_pages(table, [20], 12, 16, 4, parents=[0] * 4, new=[1] * 4)
    assert got[2].tolist() == [[-1, -1, 0], [3, 0, 4], [3, 1, 4], [3, 2, 4]]
    got = _check_pages(table, [20], 12, 16, 4, parents=[0] * 5, new=[1, 1, 1, 1, 0])
    assert got[2].tolist() == [[3, 0, 4], [3, 1, 4], [3, 2, 4], [3, 4, 4], [-1, -1, 0]]
    assert got[3].item() == 6


def test_pages_that_run_out():
    table = [[0, 1, 2, -1, -1, -1], [3, 4, 5, -1, -1, -1]]
    for pages in (6, 7, 8, 9, 30):
        _check_pages(table, [40, 48], pages, 16, 6, parents=[0, 0, 1, 1, -1], new=[30, 30, 1, 20, 17])
    _check_pages([[-1] * 6], [0], 0, 16, 6, new=[40])


def test_no_sequences():
    got = ops.cache_pages(torch.empty(0, 4, dtype=torch.int32, device="cuda"), _ints([]), 9, 16,
                          parents=_ints([-1, -1]), new=_ints([20, 1]))
    assert got[0].tolist() == [[0, 1, -1, -1], [2, -1, -1, -1]] and got[1].tolist() == [20, 1]
    assert got[3].item() == 6
    got = ops.cache_pages(torch.empty(0, 4, dtype=torch.int32, device="cuda"), _ints([]), 9, 16)
    assert got[0].shape == (0, 4) and got[2].shape == (0, 3) and got[3].item() == 9


def test_outputs_given_graphs_and_streams():
    lens, width, parents, kept, new = _random_step(3, 30, 30, 32, 700, 2)
    table = _table(lens, 32, width, 900, 3, 2)
    args = [_ints(table), _ints(lens), 900, 32, _ints(parents), _ints(kept), _ints(new)]
    want = _check_pages(table, lens, 900, 32, width, parents, kept, new)
    out = tuple(torch.full_like(t, 77) for t in want)
    got = ops.cache_pages(*args, out=out)
    assert all(a is b for a, b in zip(got, out)) and all(torch.equal(a, b) for a, b in zip(out, want))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = ops.cache_pages(*args, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    # two tables that a captured loop takes in turn: 40 tokens for every row, one after the other
    first = ops.cache_pages(*args)
    one = _ints([1] * 30)
    second = tuple(torch.empty_like(t) for t in first)
    back = tuple(torch.empty_like(t) for t in first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.cache_pages(first[0], first[1], 900, 32, new=one, out=second)
        ops.cache_pages(second[0], second[1], 900, 32, new=one, out=back)
        for a, b in zip(first, back):
            a.copy_(b)
    state = [t.tolist() for t in first]
    for _ in range(20):
        graph.replay()
    for _ in range(40):
        state = br.pages(state[0], state[1], 900, 32, new=[1] * 30)
    for g, w in zip(first, state):
        assert torch.equal(g.cpu(), torch.tensor(w, dtype=torch.int32).reshape(g.shape))


def test_table_errors_are_recorded_and_cut_down():
    table, lens = [[0, 1, -1], [2, 3, -1]], [20, 32]
    for what, change in ((5, dict(parents=[2, 0])), (5, dict(parents=[-2, 0])), (3, dict(kept=[21, 0])),
                         (3, dict(kept=[-1, 0])), (3, dict(new=[-5, 0])), (3, dict(new=[29, 0])),
                         (3, dict(new=[2 ** 31 - 1, 0])), (3, dict(lens=[49, 32])), (3, dict(lens=[-1, 0])),
                         (2, dict(table=[[0, 9, -1], [2, 3, -1]])), (2, dict(table=[[-1, 1, -1], [2, 3, -1]]))):
        a = dict(table=table, lens=lens, parents=None, kept=None, new=None)
        a.update(change)
        got = ops.cache_pages(_ints(a["table"]), _ints(a["lens"]), 9, 16, _ints(a["parents"]),
                              _ints(a["kept"]), _ints(a["new"]))
        st, info = ops.get_cache_error()
        assert st == 2 and info[1] == 36 and info[2] == what and info[3] == 0, (change, info)
        t = got[0].cpu()
        assert ((t >= -1) & (t < 9)).all()
        if "lens" not in change and "parents" not in change:           # the other row is as it should be
            assert t[1].tolist() == br.pages([table[1]], [lens[1]], 9, 16, kept=None if a["kept"] is None else [0],
                                             new=None)[0][0]


# ------------------------------------------------------------------------------------
# copies
# ------------------------------------------------------------------------------------

def _pools(pages, heads, D, page, seed):
    g = torch.Generator().manual_seed(seed)
    codes = [torch.randint(256, (pages, heads, page, D), generator=g, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.rand(pages, heads, generator=g) for _ in range(2)]
    return codes, scales


def _on_gpu(codes, scales):
    return [c.cuda().view(F8) for c in codes] + [s.cuda() for s in scales]


@pytest.mark.parametrize("n,heads,D,page,whole", [(1, 1, 64, 16, False), (5, 2, 96, 16, False),
                                                  (40, 8, 128, 64, False), (9, 3, 256, 256, True),
                                                  (700, 2, 64, 32, False), (33, 1, 192, 128, False),
                                                  (150, 8, 128, 128, True)])
def test_copies(n, heads, D, page, whole):
    r = random.Random(n)
    pages = 2 * n + 3
    order = list(range(pages))
    r.shuffle(order)
    copies = [[order[i], order[n + i], page if whole else r.randint(0, page)] for i in range(n)]
    if n > 4:                                        # one page to several, and rows that copy nothing
        copies[1][0] = copies[0][0]
        copies[2] = [-1, -1, 0]
        copies[3] = [5, -1, 3]
        copies[4][1] = copies[4][0]
    codes, scales = _pools(pages, heads, D, page, n)
    dev = _on_gpu(codes, scales)
    assert ops.cache_copy(*dev, _ints(copies)) is None
    for c, s in zip(codes, scales):
        for a, z, t in copies:
            if a >= 0 and z >= 0 and t > 0:
                c[z, :, :t], s[z] = c[a, :, :t], s[a]
    for g, w in zip(dev, codes + scales):
        assert torch.equal(g.view(w.dtype).cpu(), w)


def test_copy_errors_and_nothing_to_copy():
    codes, scales = _pools(6, 2, 64, 16, 1)
    for what, bad in ((2, [6, 1, 3]), (2, [1, 7, 3]), (3, [1, 2, 17]), (3, [1, 2, -1])):
        dev = _on_gpu(codes, scales)
        ops.cache_copy(*dev, _ints([bad, [3, 4, 5]]))
        st, info = ops.get_cache_error()
        assert st == 2 and info[1:] == [37, what, 0], info
        got = dev[0].view(torch.uint8).cpu()
        assert torch.equal(got[:4], codes[0][:4]) and torch.equal(got[4, :, :5], codes[0][3, :, :5])
    dev = _on_gpu(codes, scales)
    ops.cache_copy(*dev, torch.empty(0, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="copies"):
        ops.cache_copy(*dev, _ints([1, 2]))
    with pytest.raises(TypeError, match="copies"):
        ops.cache_copy(*dev, torch.zeros(1, 3, device="cuda"))
    assert torch.equal(dev[0].view(torch.uint8).cpu(), codes[0])


def test_copies_past_32_bit_offsets():
    heads, D, page = 8, 128, 256                     # 256 KB a page
    pages = 2 ** 32 // (heads * D * page) + 40
    k = torch.zeros(pages, heads, page, D, dtype=torch.uint8, device="cuda").view(F8)
    v = torch.zeros_like(k)
    ks, vs = torch.zeros(pages, heads, device="cuda"), torch.zeros(pages, heads, device="cuda")
    k.view(torch.uint8)[pages - 1] = 5
    v.view(torch.uint8)[2] = 9
    ks[pages - 1], vs[2] = 0.5, 0.25
    ops.cache_copy(k, v, ks, vs, _ints([[pages - 1, 1, page], [2, pages - 2, 100]]))
    assert (k.view(torch.uint8)[1] == 5).all() and (v.view(torch.uint8)[1] == 0).all()
    assert (v.view(torch.uint8)[pages - 2, :, :100] == 9).all()
    assert (v.view(torch.uint8)[pages - 2, :, 100:] == 0).all()
    assert ks[1, 3] == 0.5 and vs[pages - 2, 7] == 0.25


# ------------------------------------------------------------------------------------
# kept tokens moved together
# ------------------------------------------------------------------------------------

def _kept(c, first, counts, seed):
    r = random.Random(seed)
    return [sorted(r.sample(range(f, n), k)) for f, n, k in zip(first, c.lens, counts)]


def _check_compact(c, first, tokens, counts, stream=None):
    most = max([len(t) for t in tokens] + [1])
    padded = [t + [-9] * (most - len(t)) for t in tokens]
    kc, vc, ks, vs, table, lens = c.args(starts=False)
    assert ops.cache_compact(kc, vc, ks, vs, table, lens, _ints(first), _ints(padded), _ints(counts),
                             stream=stream) is None
    for codes, scale, g, gs in ((c.k, c.ks, kc, ks), (c.v, c.vs, vc, vs)):
        want, s = br.compact(codes, scale, c.table.tolist(), c.page, first, tokens, counts)
        assert torch.equal(gs.cpu().double().nan_to_num(-1), s.nan_to_num(-1))
        # of a page that received tokens, the slots up to the sequence's end; all others as they were
        same = torch.ones(codes.shape[0], c.page, dtype=torch.bool)
        for b, (f, n) in enumerate(zip(first, counts)):
            if n and (f + n) % c.page:
                same[c.table[b, (f + n) // c.page], (f + n) % c.page:] = False
        same = same[:, None, :, None].expand(codes.shape)
        bad = (g.cpu().double() != want) & same & ~(g.cpu().double().isnan() & want.isnan())
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    return kc, vc, ks, vs


@pytest.mark.parametrize("older,new,counts,heads,D,page", [
    ([0], [1], [1], 1, 64, 16), ([20], [8], [3], 2, 64, 16), ([15, 16, 17, 0], [9, 5, 16, 4], [4, 0, 7, 4], 2, 128, 16),
    ([100, 0], [64, 40], [9, 40], 3, 96, 32), ([250, 3], [30, 200], [11, 77], 2, 128, 64),
    ([4, 0], [1500, 700], [600, 699], 2, 64, 16), ([4], [3000], [1111], 1, 128, 128),
    ([4, 9, 0], [900, 10, 0], [333, 10, 0], 2, 256, 256), ([0, 500], [5000, 3], [2500, 1], 1, 192, 32),
    ([1], [9000], [4500], 1, 64, 64), ([3], [9000], [6000], 1, 256, 256), ([0], [5000], [4100], 1, 96, 16),
    ([60] * 90, [12] * 90, [1 + b % 12 for b in range(90)], 2, 64, 32),
])
def test_compact(older, new, counts, heads, D, page):
    c = ref.Cache(older, new, heads, D, page, seed=D + page)
    c.ks *= torch.exp(torch.randn(c.ks.shape, generator=torch.Generator().manual_seed(2)))
    _check_compact(c, older, _kept(c, older, counts, page), counts)


def test_kept_in_place_and_equal_scales():
    """Tokens that stay where they are change nothing; tokens of pages of one scale keep their codes."""
    c = ref.Cache([30, 5], [90, 60], 2, 64, 16, seed=3)
    got = _check_compact(c, [30, 5], [list(range(30, 120)), list(range(5, 65))], [90, 60])
    for g, w in zip(got, (c.k, c.v, c.ks, c.vs)):
        assert torch.equal(g.cpu().view(torch.uint8), w.view(torch.uint8))
    c.ks.fill_(0.5)
    c.vs.fill_(0.25)
    tokens = _kept(c, [30, 5], [40, 33], 4)
    kc, vc, ks, vs = _check_compact(c, [30, 5], tokens, [40, 33])
    assert (ks == 0.5).all() and (vs == 0.25).all()


def test_compact_past_32_bit_offsets():
    """Pages whose bytes lie past 4 GB of their pools."""
    heads, D, page = 8, 128, 256
    pages = 2 ** 32 // (heads * page * D) + 12
    c = ref.Cache([3], [1500], heads, D, page, seed=4, spare=0)
    n = c.pages
    far = torch.arange(pages - n, pages)
    kc = torch.zeros(pages, heads, page, D, dtype=torch.uint8, device="cuda").view(F8)
    vc = torch.zeros_like(kc)
    ks, vs = torch.zeros(pages, heads, device="cuda"), torch.zeros(pages, heads, device="cuda")
    for small, large in ((c.k, kc), (c.v, vc)):
        large.view(torch.uint8)[far.cuda()] = small.view(torch.uint8).cuda()
    ks[far.cuda()], vs[far.cuda()] = c.ks.cuda(), c.vs.cuda()
    table = torch.where(c.table >= 0, c.table + pages - n, -1)
    tokens = _kept(c, [3], [700], 5)
    ops.cache_compact(kc, vc, ks, vs, table.cuda(), _ints(c.lens), _ints([3]), _ints(tokens), _ints([700]))
    for codes, scale, g, gs in ((c.k, c.ks, kc, ks), (c.v, c.vs, vc, vs)):
        want, s = br.compact(codes, scale, c.table.tolist(), page, [3], tokens, [700])
        assert torch.equal(gs[far.cuda()].cpu().double(), s)
        got = g[far.cuda()].cpu().double()
        for j in range(703):
            assert torch.equal(got[c.table[0, j // page], :, j % page], want[c.table[0, j // page], :, j % page])
        assert (g.view(torch.uint8)[: pages - n] == 0).all()


def test_compact_of_zero_scales_and_nan_codes():
    c = ref.Cache([10], [100], 2, 64, 16, seed=5)
    c.ks[c.table[0, 2]] = 0                          # a page of zeros
    c.ks[c.table[0, 0]] = c.ks[c.table[0, 1]] = 0
    c.vs[:] = 0
    c.k.view(torch.uint8)[c.table[0, 3], :, 5] = 0x7F
    c.v.view(torch.uint8)[c.table[0, 4], :, 6] = 0xFF
    _check_compact(c, [10], [list(range(12, 100, 2))], [44])


def test_compact_on_a_stream_and_in_a_graph():
    c = ref.Cache([20, 7], [300, 50], 2, 128, 32, seed=6)
    tokens = _kept(c, [20, 7], [100, 20], 1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        want = _check_compact(c, [20, 7], tokens, [100, 20])
    kc, vc, ks, vs, table, lens = c.args(starts=False)
    args = [_ints([20, 7]), _ints([t + [0] * (100 - len(t)) for t in tokens]), _ints([100, 20])]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ops.cache_compact(kc, vc, ks, vs, table, lens, *args)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((kc, vc, ks, vs), want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_compact_errors_are_recorded():
    c = ref.Cache([20, 7], [30, 50], 2, 64, 16, seed=6)
    good = [[21, 25, 30], [8, 20, 56]]
    for what, change in ((3, dict(first=[20, -1])), (3, dict(counts=[3, 4])), (3, dict(counts=[3, -1])),
                         (3, dict(first=[20, 55])), (3, dict(lens=[50, 10 ** 6])), (6, dict(tokens=[good[0], [8, 20, 57]])),
                         (6, dict(tokens=[good[0], [6, 20, 56]])), (6, dict(tokens=[good[0], [8, 20, 20]])),
                         (6, dict(tokens=[good[0], [8, 7, 20]])), (2, dict(page=(1, 1, 10 ** 6))),
                         (2, dict(page=(1, 3, -1)))):
        a = dict(first=[20, 7], tokens=good, counts=[3, 3], lens=c.lens, page=None)
        a.update(change)
        kc, vc, ks, vs, table, lens = c.args(starts=False)
        if a["page"]:
            table[a["page"][0], a["page"][1]] = a["page"][2]
        ops.cache_compact(kc, vc, ks, vs, table, _ints(a["lens"]), _ints(a["first"]), _ints(a["tokens"]),
                          _ints(a["counts"]))
        st, info = ops.get_cache_error()
        assert st == 2 and info[1:] == [38, what, 1], (change, info)
        want, s = br.compact(c.k, c.ks, c.table.tolist(), 16, [20], [good[0]], [3])
        mine = c.table[0, :4].long()                 # the other sequence is as it should be
        assert torch.equal(ks.cpu().double()[mine], s[mine])
        assert torch.equal(kc.cpu().double()[mine][1, :, :7], want[mine][1, :, :7])


def test_compact_refusals():
    c = ref.Cache([20, 7], [30, 50], 2, 64, 16, seed=6)
    args = c.args(starts=False)
    first, tokens, counts = _ints([20, 7]), _ints([[21], [8]]), _ints([1, 1])
    for bad, error in (((None, tokens, counts), TypeError), ((first, tokens, None), TypeError),
                       ((first, tokens[0], counts), ValueError), ((first, tokens.long(), counts), TypeError),
                       ((first[:1], tokens, counts), ValueError), ((first, tokens, counts.cpu()), ValueError)):
        with pytest.raises(error):
            ops.cache_compact(*args, *bad)
    ops.cache_compact(*args, first, tokens[:, :0].contiguous(), counts * 0)


def test_pages_refusals():
    table, lens = _ints([[0, 1], [2, 3]]), _ints([20, 20])
    with pytest.raises(ValueError, match="out"):
        ops.cache_pages(table, lens, 9, 16, out=(table,))
    with pytest.raises(ValueError, match="followed"):
        ops.cache_pages(table, lens, 9, 16, new=_ints([1, 1, 1]))
    with pytest.raises(ValueError, match="kept"):
        ops.cache_pages(table, lens, 9, 16, parents=_ints([0]), kept=_ints([1, 2]))
    with pytest.raises(TypeError):
        ops.cache_pages(table.long(), lens, 9, 16)
    fresh = ops.cache_pages(table, lens, 9, 16)
    for i, over in ((0, table), (1, lens)):
        out = list(fresh)
        out[i] = over
        with pytest.raises(ops.B2BError, match="UNSUPPORTED"):
            ops.cache_pages(table, lens, 9, 16, out=out)
    out = list(fresh)
    out[3] = out[1][:1]
    with pytest.raises(ops.B2BError, match="UNSUPPORTED"):
        ops.cache_pages(table, lens, 9, 16, out=out)
    for bad in (dict(page_size=24), dict(pages=-1), dict(page_size=8), dict(pages=2 ** 31)):
        a = dict(pages=9, page_size=16)
        a.update(bad)
        with pytest.raises(ops.B2BError):
            ops.cache_pages(table, lens, a["pages"], a["page_size"])
    with pytest.raises(ops.B2BError, match="UNSUPPORTED"):
        ops.cache_pages(table, lens, 9, 16, parents=_ints([-1] * 4097))
