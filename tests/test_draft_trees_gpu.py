"""The operators of drafted and branching sequences run together, as the example does: pages, copies, the
append, tree attention and the kept path, step after step, against 64-bit forms over what is cached."""
import pytest
import torch

import branch_ref as br
import decoder_ref as ref
from gemm_conv_chains_gb300 import ops

pytestmark = pytest.mark.gpu
RTOL = 2e-2        # the framework's bar for bf16 chains, |gpu - ref| <= RTOL * max(1, |ref|)


def _round(t):
    return t.to(torch.bfloat16).double()


def _cache(rows, new, ex):
    """What the GPU's cache and page table hold, as the references take it."""
    lens = rows.lens.tolist()
    c = ref.Cache([n - m for n, m in zip(lens, new)], new, ex.KV_HEADS, ex.HEAD, ex.PAGE)
    c.k, c.v, c.ks, c.vs = (t.cpu() for t in rows.pool())
    c.table = rows.table.cpu()
    return c


def _want(block, c, x, ex):
    """The block over one tree per sequence in 64 bits, on the cached keys and values."""
    w = {k: getattr(block, k).cpu().double() for k in ("wq", "wo", "w0", "w1")}
    x = x.cpu().double()
    depth = torch.tensor(ex.DEPTH)
    positions = torch.cat([a + depth for a in c.older])
    q = ref.turn(_round(x @ w["wq"]).view(-1, ex.HEADS, ex.HEAD), block.table.cpu().double()[positions], "half")
    seen = br.ancestors(ex.PARENTS)
    a, _ = br.tree_attention(c, _round(q), [seen] * len(c.new), ex.HEAD ** -0.5)
    x = _round(x + _round(_round(a).reshape(-1, ex.WIDTH) @ w["wo"]))
    h = x @ w["w0"]
    h = _round(h * ((h + 3).clamp(0, 6) / 6))
    return _round(x + _round(h @ w["w1"]))


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ops.lib()
    ops.get_cache_error()
    yield
    st, info = ops.get_cache_error()
    assert st == 0, f"cache error word left set: {st} {info}"


def test_trees_and_beams_step_after_step():
    from examples import draft_trees as ex
    B, new = 5, [40, 3, 32, 61, 17]
    block = ex.TreeBlock(B, positions=200, seed=3)
    rows = ex.Rows(B, 60, 6)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(sum(new), ex.WIDTH, generator=g).bfloat16().cuda()
    block.prompts(x, rows, torch.tensor(new, dtype=torch.int32, device="cuda"), max(new))
    kept = rows.lens.clone()
    room = torch.full((B,), ex.NODES, dtype=torch.int32, device="cuda")
    history = [None] * B                             # the values that each sequence holds
    for step in range(6):
        # two beams branch off the first, another off the third for some of its tokens
        parents = None
        if step in (1, 4):
            parents = [0, 0, 2, 2, 0]
            kept = kept[torch.tensor(parents, device="cuda")]
            kept[3] -= 5
            history = [history[p] for p in parents]
        before = rows.table.tolist(), rows.lens.tolist()
        want = br.pages(*before, 60, ex.PAGE, parents, kept.tolist(), [ex.NODES] * B)
        rows.step(room, kept, None if parents is None else torch.tensor(parents, dtype=torch.int32, device="cuda"))
        assert rows.table.tolist() == want[0] and rows.lens.tolist() == want[1]
        assert rows.left.item() == want[3][0] >= 0
        c = _cache(rows, [ex.NODES] * B, ex)
        for b, n in enumerate(kept.tolist()):        # what a row held it still holds, copies included
            k, v = c.values(b, n)
            if history[b] is not None:
                for got, was in zip((k, v), history[b]):
                    assert torch.equal(got, was[:, :n])
        x = torch.randn(B * ex.NODES, ex.WIDTH, generator=g).bfloat16()
        y = block.drafts(x.cuda(), rows)
        c = _cache(rows, [ex.NODES] * B, ex)
        want = _want(block, c, x, ex)
        err = (y.cpu().double().view(-1, ex.WIDTH) - want).abs()
        assert (err <= RTOL * want.abs().clamp_min(1)).all(), err.max()
        path, count = block.accept(y)
        first = (rows.lens - ex.NODES).tolist()
        paths, counts = path.tolist(), count.tolist()
        for p, n in zip(paths, counts):              # a path of the tree
            assert p[0] == 0 and all(ex.PARENTS[p[i]] == p[i - 1] for i in range(1, n))
        tokens = [[f + i for i in p] for f, p in zip(first, paths)]
        kept = block.keep(rows, path, count)
        assert kept.tolist() == [f + n for f, n in zip(first, counts)]
        after = _cache(rows, [ex.NODES] * B, ex)
        for codes, scale, got, got_scale in ((c.k, c.ks, after.k, after.ks), (c.v, c.vs, after.v, after.vs)):
            want, s = br.compact(codes, scale, c.table.tolist(), ex.PAGE, first, tokens, counts)
            assert torch.equal(got_scale.double(), s)
            for b, n in enumerate(kept.tolist()):
                for j in range(n):
                    at, slot = c.table[b, j // ex.PAGE], j % ex.PAGE
                    assert torch.equal(got[at, :, slot].double(), want[at, :, slot])
        history = [after.values(b, n) for b, n in enumerate(kept.tolist())]


def test_the_example_runs(capsys, monkeypatch):
    from examples import draft_trees as ex
    monkeypatch.setattr("sys.argv", ["draft_trees.py", "--batch", "6", "--prompt", "70", "--steps", "9"])
    ex.main()
    assert "tokens kept" in capsys.readouterr().out


def test_a_step_in_a_graph():
    """Two steps captured: pages into the other table and back, no call waits for the host."""
    from examples import draft_trees as ex
    B, new = 4, [20, 33, 1, 64]
    block, rows = ex.TreeBlock(B, positions=300, seed=5), ex.Rows(B, 80, 10)
    g = torch.Generator().manual_seed(6)
    x = torch.randn(sum(new), ex.WIDTH, generator=g).bfloat16().cuda()
    block.prompts(x, rows, torch.tensor(new, dtype=torch.int32, device="cuda"), max(new))
    room = torch.full((B,), ex.NODES, dtype=torch.int32, device="cuda")
    kept = rows.lens.clone()
    drafted = torch.randn(2, B * ex.NODES, ex.WIDTH, generator=g).bfloat16().cuda()

    def two_steps():
        ys = []
        for i in range(2):
            rows.step(room, kept)
            y = block.drafts(drafted[i], rows)
            kept.copy_(block.keep(rows, *block.accept(y)))
            ys.append(y)
        return ys

    start = [t.clone() for t in (*rows.pool(), rows.table, rows.lens, kept)]
    live = [*rows.pool(), rows.table, rows.lens, kept]
    eager = [y.clone() for _ in range(2) for y in two_steps()]
    for t, s in zip(live, start):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        captured = two_steps()
    for t, s in zip(live, start):
        t.copy_(s)
    replayed = []
    for _ in range(2):
        graph.replay()
        replayed += [y.clone() for y in captured]
    torch.cuda.synchronize()
    for a, b in zip(eager, replayed):
        assert torch.equal(a, b)
