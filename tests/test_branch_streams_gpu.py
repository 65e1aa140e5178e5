"""The operators of drafted and branching sequences from several streams, threads and graphs: where
their outputs lie, workspaces that calls and graphs share one after the other, calls at once."""
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


def _tree(seed, older, new, heads, group, D):
    """(arguments of the attention of a drafted tree, its rows and masks first)"""
    c = ref.Cache(older, new, heads, D, 64, seed=seed, fill=0x7F)
    blocks = [br.ancestors(br.tree(n, seed + b, 4)) for b, n in enumerate(new)]
    q = torch.randn(c.T, heads * group, D, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
    return [q, br.words(blocks).cuda(), *c.args()]


# the split kernel, cut; the wide one over cut and over whole units
TREES = [([1200, 90], [9, 30], 2, 4, 128), ([2600, 700], [60, 33], 8, 2, 128),
         ([400, 120, 0, 800, 300, 64, 1, 511], [30, 12, 40, 7, 25, 32, 40, 1], 4, 3, 128)]


def _pool(t):
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


def test_outputs_come_from_the_memory_of_the_stream_that_writes_them():
    side = torch.cuda.Stream()
    tree = _tree(1, *TREES[0])
    table, lens = torch.full((200, 8), -1, dtype=torch.int32, device="cuda"), _ints([0] * 200)
    calls = [lambda s: (ops.cache_tree_attention(*tree, stream=s),),
             lambda s: ops.cache_pages(table, lens, 50, 16, new=_ints([0] * 200), stream=s)]
    torch.cuda.synchronize()
    for call in calls:
        for stream, pool in ((side, side.cuda_stream), (side.cuda_stream, side.cuda_stream), (None, 0), (0, 0)):
            out = call(stream)
            torch.cuda.synchronize()
            assert {_pool(t) for t in out} == {pool}
        with torch.cuda.stream(side):
            assert {_pool(t) for t in call(None)} == {side.cuda_stream}


@pytest.mark.parametrize("at", range(len(TREES)))
def test_graphs_and_calls_share_a_workspace(at):
    """Two graphs and a direct call, on other lengths each, in the memory of one workspace."""
    older, new, heads, group, D = TREES[at]
    trees = [_tree(s, [max(0, n - 7 * s) for n in older], new, heads, group, D) for s in (1, 2)]
    T, Hq = trees[0][0].shape[:2]
    size = max(ops.cache_tree_attention_workspace(T, Hq, *t[2:]) for t in trees)
    space = torch.full((max(size, 16),), 0xA5, dtype=torch.uint8, device="cuda")
    want = [ops.cache_tree_attention(*t) for t in trees]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    graphs = []
    for t, o in zip(trees, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            ops.cache_tree_attention(*t, out=o, workspace=space)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graphs[0].replay()
        graphs[1].replay()
        again = ops.cache_tree_attention(*trees[0], workspace=space)
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(again, want[0])


def test_threads_on_streams_of_their_own():
    """Each thread's step: room, copies, the tree's attention, the accepted tokens moved together."""
    wrong, failed = [], []

    def step(seed, kept):
        c = ref.Cache([700, 90], [60, 33], 4, 128, 32, seed=seed)
        tree = _tree(seed, *TREES[1])
        pools = [c.k.cuda(), c.v.cuda(), c.ks.cuda(), c.vs.cuda()]
        table, lens = c.table.cuda(), _ints(c.lens)
        tokens = _ints([[700 + 2 * i for i in range(kept)], [90 + i for i in range(kept)]])
        torch.cuda.synchronize()

        def run():
            mine = [p.clone() for p in pools]
            out = ops.cache_tree_attention(*tree)
            ops.cache_compact(*mine, table, lens, _ints([700, 90]), tokens, _ints([kept, kept]))
            # both branch off twice: everything is shared, and each copy's page is the next free one
            rows = ops.cache_pages(table, _ints([700 + kept, 90 + kept]), mine[0].shape[0] + 64, 32,
                                   _ints([0, 0, 1, 1]), None, _ints([3, 3, 3, 3]))
            return [out, *[m.view(torch.uint8) for m in mine], *rows]
        return run

    runs = [step(s, k) for s, k in ((3, 11), (4, 30), (5, 20))]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()

    def work(run, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(15):
                    for a, b in zip(run(), want):
                        if not torch.equal(a, b):
                            wrong.append(a.shape)
        except BaseException as e:                     # raised again below
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(runs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and not wrong, (failed, wrong[:3])


def test_padded_batches():
    """Rows of a batch that hold no sequence: zero lengths, tables of -1, no tokens; nothing of theirs moves."""
    c = ref.Cache([300, 0, 40], [10, 0, 6], 2, 64, 16, seed=2)
    assert c.table[1].eq(-1).all()
    args = c.args()
    blocks = [br.ancestors(br.tree(n, b, 4)) for b, n in enumerate(c.new) if n]
    q = torch.randn(c.T + 5, 4, 64, generator=torch.Generator().manual_seed(2)).half().cuda()
    masks = torch.cat([br.words(blocks), torch.full((5, 1), -1)]).cuda()
    out = torch.full((c.T + 5, 4, 64), 3.0, dtype=torch.float16, device="cuda")
    ops.cache_tree_attention(q, masks, *args, out=out)
    assert (out[c.T:] == 3.0).all()
    assert torch.equal(out[: c.T], ops.cache_tree_attention(q[: c.T], masks[: c.T], *args))
    pools = [t.clone() for t in args[:4]]
    ops.cache_compact(*args[:6], _ints([300, 0, 40]), _ints([[301, 305], [0, 0], [41, 43]]), _ints([2, 0, 0]))
    used = c.table[0].long().cuda()
    for now, was in zip(args[:4], pools):
        now, was = now.view(torch.uint8), was.view(torch.uint8)
        others = torch.ones(now.shape[0], dtype=torch.bool, device="cuda")
        others[used[used >= 0]] = False
        assert torch.equal(now[others], was[others])
    table, lens, copies, left = ops.cache_pages(args[4], _ints([302, 0, 40]), c.pages, 16, _ints([0, -1, -1]))
    assert (table[1:] == -1).all() and lens.tolist() == [302, 0, 0] and (copies[:, :2] == -1).all()
    assert left.item() == c.pages - (302 + 15) // 16
