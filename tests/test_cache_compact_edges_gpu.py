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
