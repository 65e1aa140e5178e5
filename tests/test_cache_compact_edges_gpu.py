"""Kept tokens moved together: what is left where a token is refused, sequences that share pages."""
import threading

import pytest
import torch

from gemm_conv_chains_gb300 import ops

import branch_ref as br
import decoder_ref as ref

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


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (96, 32)])
@pytest.mark.parametrize("what", ["all of a page", "some of a page", "behind older tokens", "a page that is none"])
def test_what_a_refused_token_leaves(what, D, page):
    """It is recorded, its slot keeps the token that it had, with the page's scale as that token's: the
    result is that of the same call with the slot's own token in its place."""
    first = page if what != "behind older tokens" else page - 3
    c = ref.Cache([first], [5 * page], 2, D, page, seed=D)
    c.ks *= torch.exp(torch.randn(c.ks.shape, generator=torch.Generator().manual_seed(1)))
    tokens = list(range(first + 1, first + 4 * page, 2))           # two pages of them
    meant = list(tokens)
    refused = {"all of a page": range(page), "some of a page": (1, 4, page - 1, page + 2),
               "behind older tokens": range(3), "a page that is none": ()}[what]
    for i in refused:
        tokens[i], meant[i] = -5, first + i
    table = c.table.clone()
    if what == "a page that is none":
        gone = meant[page + 2] // page                             # some of the second page's come from it
        table[0, gone] = c.pages
        for i, t in enumerate(meant):
            if t // page == gone:
                meant[i] = first + i
    kc, vc, ks, vs, _, lens = c.args(starts=False)
    ops.cache_compact(kc, vc, ks, vs, table.cuda(), lens, _ints([first]), _ints([tokens]), _ints([len(tokens)]))
    st, info = ops.get_cache_error()
    assert st == 2 and info[1] == 38 and info[2] == (2 if what == "a page that is none" else 6)
    end = first + len(tokens)
    for codes, scale, g, gs in ((c.k, c.ks, kc, ks), (c.v, c.vs, vc, vs)):
        want, s = br.compact(codes, scale, c.table.tolist(), page, [first], [meant], [len(meant)])
        assert bool((gs.cpu().double() == s).all())
        got = g.cpu().double()
        for j in range(end):
            at = int(c.table[0, j // page])
            assert bool((got[at, :, j % page] == want[at, :, j % page]).all()), j


def test_the_first_call_of_a_thread_in_a_graph():
    """Whatever a thread's first call asks of the device, it may ask while a graph is captured."""
    c = ref.Cache([4], [5000], 1, 64, 64, seed=2)
    tokens = list(range(5, 5004, 3))
    kc, vc, ks, vs, table, lens = c.args(starts=False)
    lists = _ints([4]), _ints([tokens]), _ints([len(tokens)])
    before = [t.clone() for t in (kc, vc, ks, vs)]
    ops.cache_compact(kc, vc, ks, vs, table, lens, *lists)
    want = [t.clone() for t in (kc, vc, ks, vs)]
    for t, b in zip((kc, vc, ks, vs), before):
        t.copy_(b)
    graph, failed = torch.cuda.CUDAGraph(), []

    def capture():
        try:
            with torch.cuda.graph(graph):
                ops.cache_compact(kc, vc, ks, vs, table, lens, *lists)
        except Exception as e:                       # noqa: BLE001 (shown by the assertion below)
            failed.append(e)

    torch.cuda.synchronize()
    thread = threading.Thread(target=capture)
    thread.start()
    thread.join()
    assert not failed, failed
    graph.replay()
    torch.cuda.synchronize()
    for got, w in zip((kc, vc, ks, vs), want):
        assert bool((got.view(torch.uint8) == w.view(torch.uint8)).all())


@pytest.mark.parametrize("D,page,n", [(64, 16, 100), (128, 64, 700), (256, 32, 96)])
def test_evicting_from_one_of_two_that_share_pages(D, page, n):
    """A branch gets pages of its own (a row of no parent, its pages copied) before it loses tokens: the
    other branch keeps every byte, and the evicted one has what it would have had alone."""
    c = ref.Cache([0], [n], 2, D, page, seed=D, spare=-(-n // page) + 2)
    c.ks *= torch.exp(torch.randn(c.ks.shape, generator=torch.Generator().manual_seed(1)))
    kc, vc, ks, vs, table, lens = c.args(starts=False)
    pool = kc, vc, ks, vs
    table, lens, copies, left = ops.cache_pages(table, lens, c.pages, page, _ints([0, 0]))
    assert bool((table[0] == table[1]).all()) and bool((copies[:, 0] == -1).all())
    mine = [t.clone() for t in pool]
    # row 2: room for all that row 1 has; then row 1's pages into it
    table, lens, copies, left = ops.cache_pages(table, lens, c.pages, page, _ints([0, 1, -1]), None, _ints([0, 0, n]))
    assert left.item() >= 0
    pages = -(-n // page)
    each = [min(page, n - j * page) for j in range(pages)]
    ops.cache_copy(*pool, torch.stack([table[1, :pages], table[2, :pages], _ints(each)], 1).contiguous())
    tokens = [j for j in range(n) if j < 4 or j % 3 == 1]
    ops.cache_compact(*pool, table, lens, _ints([n, n, 0]), _ints([tokens] * 3), _ints([0, 0, len(tokens)]))
    kept = _ints([n, len(tokens)])
    table, lens, copies, left = ops.cache_pages(table, lens, c.pages, page, _ints([0, 2]), kept)
    assert lens.tolist() == kept.tolist() and bool((copies[:, 0] == -1).all())
    assert left.item() == c.pages - pages - -(-len(tokens) // page)
    for t, b, codes, scale, s in ((kc, mine[0], c.k, c.ks, ks), (vc, mine[1], c.v, c.vs, vs)):
        own = table[0, :pages].long()
        assert bool((t.view(torch.uint8)[own] == b.view(torch.uint8)[own]).all())
        assert bool((s.cpu()[own.cpu()] == scale[own.cpu()]).all())
        want, ws = br.compact(codes, scale, c.table.tolist(), page, [0], [tokens], [len(tokens)])
        got, gs = t.cpu().double(), s.cpu().double()
        for j in range(len(tokens)):
            at, as_at = int(table[1, j // page]), int(c.table[0, j // page])
            assert at not in own.tolist() and bool((gs[at] == ws[as_at]).all())
            assert bool((got[at, :, j % page] == want[as_at, :, j % page]).all()), j
