"""Attention of drafted trees over the paged e4m3 cache, against its 64-bit form.  Allowed errors
follow from the stated roundings: fp32 arithmetic, fp16 probabilities, one rounding of the output."""
import math
import random

import pytest
import torch

from gemm_conv_chains_gb300 import ops

import branch_ref as br
import decoder_ref as ref
from decoder_ref import TINY, UNIT

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ops.lib()
    ops.get_cache_error()
    yield
    st, info = ops.get_cache_error()
    assert st == 0, f"cache error word left set: {st} {info}"


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def _blocks(new, seed, spread=4):
    return [br.ancestors(br.tree(n, seed + b, spread)) if n else torch.zeros(0, 0, dtype=torch.bool)
            for b, n in enumerate(new)]


def _check(got, c, q, blocks, scale, **kw):
    want, tol = br.tree_attention(c, q, blocks, scale, **kw)
    tol = tol + UNIT[q.dtype] * (want.abs() + tol) + TINY[q.dtype]
    got = got.cpu().double()
    assert torch.equal(got.isnan(), want.isnan())
    bad = ~((got - want).abs() <= tol) & ~want.isnan()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}; worst {((got - want).abs() - tol).nan_to_num().max()}, " \
                          f"first {bad.nonzero()[:3].tolist()}"


def _run(c, q, blocks, **kw):
    width = kw.pop("width", None)
    return ops.cache_tree_attention(q, br.words([b for b in blocks if b.numel()], width).cuda(), *c.args(), **kw)


# older tokens, drafted tokens, kv heads, query heads on each, head size, page size
SHAPES = [
    ([0], [1], 1, 1, 64, 16), ([199], [8], 4, 1, 64, 16), ([15, 16, 17, 255], [3, 1, 9, 2], 2, 4, 128, 16),
    ([1000, 3, 513, 64], [8, 2, 7, 8], 2, 1, 128, 64), ([700, 0, 40], [16, 5, 1], 1, 2, 128, 32),
    ([300, 2, 900], [33, 17, 40], 2, 5, 96, 32), ([77, 511], [5, 21], 2, 3, 192, 128),
    ([530, 1040], [12, 13], 1, 8, 256, 256), ([100, 7, 0], [63, 64, 65], 2, 2, 64, 64),
    ([1600, 31], [7, 2], 2, 1, 256, 32), ([90, 1100], [130, 9], 1, 5, 128, 16),
    ([0, 33, 800], [150, 0, 70], 2, 2, 64, 32), ([5, 2000], [200, 100], 4, 4, 128, 64),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("older,new,heads,group,D,page", SHAPES)
def test_trees(dt, older, new, heads, group, D, page):
    """Every head size and row tile; whatever no token was written to is NaN; strided query rows."""
    c = ref.Cache(older, new, heads, D, page, seed=D + len(older), fill=0x7F)
    blocks = _blocks(new, D)
    Hq = heads * group
    rows = _randn(D, c.T, Hq + 2, D).to(DT[dt])
    q = rows.cuda()[:, 1: 1 + Hq]
    out = _run(c, q, blocks)
    _check(out, c, rows[:, 1: 1 + Hq], blocks, D ** -0.5)
    assert torch.equal(out, _run(c, q, blocks))


@pytest.mark.parametrize("group,D", [(1, 64), (4, 128), (8, 96), (2, 256)])
def test_any_set_of_new_tokens(group, D):
    """Masks that are no trees: later tokens seen, a row's own not, none at all, bits past the end."""
    older, new = [0, 37, 0, 500, 16], [5, 20, 70, 33, 1]
    c = ref.Cache(older, new, 2, D, 16, seed=3, fill=0xFF)
    g = torch.Generator().manual_seed(5)
    blocks = [torch.rand(n, n, generator=g) < 0.3 for n in new]
    blocks[0][2] = False                             # nothing to see at all: no older tokens
    blocks[2][64] = False
    blocks[3][7] = False                             # only older tokens
    blocks[4][0] = False
    q = _randn(1, c.T, 2 * group, D).bfloat16()
    masks = br.words(blocks, 3)
    for at, n in zip(c.starts.tolist(), new):        # bits from n on are no tokens
        for w in range(3):
            bits = max(0, min(64, n - 64 * w))
            if bits < 64:
                masks[at: at + n, w] |= -1 << bits
    out = ops.cache_tree_attention(q.cuda(), masks.cuda(), *c.args())
    _check(out, c, q, blocks, D ** -0.5)
    assert (out[2] == 0).all() and (out[5 + 20 + 64] == 0).all()


def test_a_chain_is_the_causal_attention():
    """A mask of all earlier new tokens gives cache_attention's own numbers."""
    for older, new, group in [([100, 7, 900], [4, 3, 5], 2), ([800, 0], [8, 1], 1), ([60], [30], 1)]:
        c = ref.Cache(older, new, 2, 128, 32, seed=1)
        q = _randn(2, c.T, 2 * group, 128).half().cuda()
        blocks = [torch.ones(n, n).tril().bool() for n in new]
        assert torch.equal(_run(c, q, blocks), ops.cache_attention(q, *c.args()))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("softcap,bias", [(20.0, False), (0.0, True), (5.0, True)])
@pytest.mark.parametrize("older,new,heads,group,D,page", [SHAPES[2], SHAPES[5], SHAPES[7], SHAPES[9],
                                                          SHAPES[8], SHAPES[12]])
def test_cap_and_bias(dt, softcap, bias, older, new, heads, group, D, page):
    c = ref.Cache(older, new, heads, D, page, seed=D, fill=0x7F)
    blocks = _blocks(new, 11)
    Hq = heads * group
    q = (_randn(D + 1, c.T, Hq, D) * 3).to(DT[dt])
    slopes = torch.rand(Hq, generator=torch.Generator().manual_seed(2)) * 0.3 if bias else None
    depth = torch.cat([b.sum(-1) - 1 for b in blocks]).int()
    at = depth + torch.repeat_interleave(torch.tensor(older), torch.tensor(new)).int()
    for positions in (at, None):
        out = _run(c, q.cuda(), blocks, softcap=softcap, slopes=None if slopes is None else slopes.cuda(),
                   positions=None if positions is None else positions.cuda())
        _check(out, c, q, blocks, D ** -0.5, softcap=softcap, slopes=slopes, positions=positions)


def test_nans_of_hidden_tokens_stay_hidden():
    """A NaN key or value, an infinite score or a page's NaN scale reaches the rows that see it only."""
    for group, D in ((1, 64), (4, 128), (9, 128), (4, 192)):
        c = ref.Cache([40, 700], [40, 20], 2, D, 16, seed=8)
        blocks = _blocks(c.new, 21, spread=9)
        # new token 5 of the first sequence: its keys; 9: its values; all of slots 48 .. 63: the scale
        for tok, pool in ((5, c.k), (9, c.v)):
            at = 40 + tok
            pool.view(torch.uint8)[c.table[0, at // 16], 1, at % 16, 3] = 0x7F
        q = _randn(3, c.T, 2 * group, D).half()
        q[45, 0, 0] = math.inf
        out = _run(c, q.cuda(), blocks).cpu()
        want, _ = br.tree_attention(c, q, blocks, D ** -0.5)
        hit = blocks[0][:, 5]
        nan = out.isnan()
        for i in range(40):
            heads_nan = nan[i, group:].any(-1).any(-1)
            assert bool(heads_nan) == bool(hit[i] | blocks[0][i, 9]), i
            if hit[i]:
                assert nan[i, group:].all()
            if i != 45 and not hit[i]:
                assert torch.equal(nan[i], want[i].isnan())
        assert nan[45, 0].all() and not nan[45, 1:].any() or group == 1 and nan[45, 0].all()
        assert not nan[40:45].any() and not nan[46:].any()


def test_even_rows_without_starts_given_out_and_workspace():
    c = ref.Cache([1500, 3], [6, 6], 2, 128, 64, seed=4)
    blocks = _blocks(c.new, 4)
    q = _randn(5, 12, 8, 128).bfloat16()
    args = c.args(starts=False)
    masks = br.words(blocks).cuda()
    n = ops.cache_tree_attention_workspace(12, 8, *args)
    assert n > 0
    out = torch.full((12, 8, 128), 7.0, device="cuda").bfloat16()
    work = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    got = ops.cache_tree_attention(q.cuda(), masks, *args, out=out, workspace=work)
    assert got is out
    _check(out, c, q, blocks, 128 ** -0.5)
    with pytest.raises(ops.B2BError, match="SHAPE"):
        ops.cache_tree_attention(q.cuda(), masks, *args, workspace=work[:16])


def test_rows_of_no_sequence_stay_as_they_are():
    c = ref.Cache([100, 30], [7, 9], 2, 64, 16, seed=6)
    blocks = _blocks(c.new, 6)
    q = _randn(6, 20, 4, 64).half()
    masks = torch.full((20, 1), -1, dtype=torch.int64)
    masks[:16] = br.words(blocks)
    out = torch.full((20, 4, 64), 3.0, device="cuda").half()
    ops.cache_tree_attention(q.cuda(), masks.cuda(), *c.args(), out=out)
    _check(out[:16], c, q[:16], blocks, 0.125)
    assert (out[16:] == 3).all()


@pytest.mark.parametrize("B,most", [(40, 3), (150, 9), (300, 2)])
def test_many_sequences(B, most):
    r = random.Random(B)
    older = [r.randint(0, 90) for _ in range(B)]
    new = [0 if r.random() < 0.2 else r.randint(1, most) for _ in range(B)]
    new[0] = most
    for b, n in ((1, 1500), (B // 2, 900), (B - 2, 2100)):
        older[b], new[b] = n, max(new[b], 1)
    c = ref.Cache(older, new, 2, 64, 32, seed=B, fill=0x7F)
    blocks = _blocks(new, B)
    q = _randn(B, c.T, 6, 64).half()
    out = _run(c, q.cuda(), blocks)
    _check(out, c, q, blocks, 0.125)


# Enough rows and room for the kernel that takes wide trees (256 query rows per block, contexts cut in
# pieces): uncut units beside cut ones, row tiles of one row, masks of several words, most new tokens.
WIDE = [
    ([1500, 7, 0, 300], [40, 33, 64, 1], 2, 4, 64, 32), ([2000, 100], [65, 128], 1, 2, 96, 16),
    ([3000], [257], 1, 1, 128, 64), ([1100, 1, 5000], [384, 70, 200], 1, 3, 128, 128),
    ([1300, 40], [100, 0], 4, 8, 64, 256), ([900, 600, 2, 1200, 0], [70, 3, 90, 33, 12], 2, 5, 128, 16),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("older,new,heads,group,D,page", WIDE)
def test_wide_trees(dt, older, new, heads, group, D, page):
    c = ref.Cache(older, new, heads, D, page, seed=D + len(older), fill=0xFF)
    assert max(new) * group > 64 and c.table.shape[1] * page > 1024
    blocks = _blocks(new, D, 11)
    Hq = heads * group
    rows = _randn(D, c.T, Hq + 1, D).to(DT[dt])
    q = rows.cuda()[:, :Hq]
    out = _run(c, q, blocks)
    _check(out, c, rows[:, :Hq], blocks, D ** -0.5)
    assert torch.equal(out, _run(c, q, blocks))
    back = _run(c, (-rows).cuda()[:, :Hq], blocks, scale=-D ** -0.5)
    assert torch.equal(out, back)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("older,new,heads,group,D,page", WIDE)
def test_wide_trees_with_cap_and_bias(dt, older, new, heads, group, D, page):
    c = ref.Cache(older, new, heads, D, page, seed=D, fill=0x7F)
    blocks = _blocks(new, 5)
    Hq = heads * group
    q = (_randn(D + 1, c.T, Hq, D) * 3).to(DT[dt])
    slopes = torch.rand(Hq, generator=torch.Generator().manual_seed(2)) * 0.3
    depth = torch.cat([b.sum(-1) - 1 for b in blocks if b.numel()]).int()
    at = depth + torch.repeat_interleave(torch.tensor(older), torch.tensor(new)).int()
    out = _run(c, q.cuda(), blocks, softcap=20.0, slopes=slopes.cuda(), positions=at.cuda())
    _check(out, c, q, blocks, D ** -0.5, softcap=20.0, slopes=slopes, positions=at)


def test_fp16_outputs_lose_their_own_rounding_only():
    """Over all rows, the error is that of rounding the exact result to fp16: fp32 sums and 22 bits of
    each probability leave less than a tenth of it (P in 11 bits alone would add as much again)."""
    for older, new, heads, group, D in (([3000, 500], [60, 33], 2, 4, 128), ([1500], [80], 2, 2, 64),
                                        ([700, 1200], [90, 12], 2, 3, 96), ([900], [12], 2, 2, 128)):
        c = ref.Cache(older, new, heads, D, 32, seed=D)
        blocks = _blocks(new, D)
        q = (_randn(D, c.T, heads * group, D) * 0.5).half()
        out = _run(c, q.cuda(), blocks).cpu().double()
        want, _ = br.tree_attention(c, q, blocks, D ** -0.5)
        assert (out - want).norm() <= 1.1 * (want.half().double() - want).norm()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 128])
def test_wide_trees_whose_scores_and_scales_grow(dt, D):
    """Every few tokens larger than all before them, in either half of a key tile: references move again and
    again, P and the sums that are there already are scaled; value scales far apart, some zero."""
    c = ref.Cache([1500, 900], [70, 40], 2, D, 16, seed=6)
    g = torch.Generator().manual_seed(9)
    for b in range(2):
        n = -(-c.lens[b] // 16)
        ids = c.table[b, :n].long()
        c.ks[ids] *= torch.exp2(torch.linspace(-4, 6, n))[:, None]
        c.vs[ids] *= torch.exp2(torch.rand(n, 1, generator=g) * 24 - 12)
        c.vs[ids[5]] = 0
    blocks = _blocks(c.new, 3)
    q = _randn(8, c.T, 6, D).to(DT[dt])
    out = _run(c, q.cuda(), blocks)
    _check(out, c, q, blocks, D ** -0.5)


def test_wide_sets_that_hide_and_nans_that_are_hidden():
    """Rows that see no new token or nothing at all; NaN codes of new tokens reach who sees them only."""
    for D, page in ((64, 16), (128, 64), (96, 32)):
        older, new = [1200, 0, 700], [90, 70, 80]
        c = ref.Cache(older, new, 2, D, page, seed=4, fill=0x7F)
        g = torch.Generator().manual_seed(7)
        blocks = [torch.rand(n, n, generator=g) < 0.2 for n in new]
        blocks[1][5], blocks[1][69], blocks[0][3] = False, False, False
        for tok, pool in ((10, c.k), (50, c.v), (79, c.v)):
            at = older[2] + tok
            pool.view(torch.uint8)[c.table[2, at // page], 1, at % page, 9] = 0x7F
        q = _randn(3, c.T, 6, D).bfloat16()
        out = _run(c, q.cuda(), blocks).cpu()
        assert (out[90 + 5] == 0).all() and (out[90 + 69] == 0).all()
        want, tol = br.tree_attention(c, q, blocks, D ** -0.5)
        assert torch.equal(out.isnan(), want.isnan())
        assert out.isnan().any() and not out[:160].isnan().any()
        tol = tol + UNIT[q.dtype] * (want.abs() + tol) + TINY[q.dtype]
        assert (((out.double() - want).abs() <= tol) | want.isnan()).all()


# Shapes that go to the wide kernel: cut and whole units; of one row tile, whose key tiles two softmaxes
# share, and of two; both in one sequence.
TAKEN = [
    (True, [2600, 700], [60, 33], 8, 2, 128, 64), (True, [2600, 900], [64, 20], 8, 4, 64, 16),
    (True, [1800, 5, 0, 2000], [70, 128, 90, 1], 4, 3, 96, 32), (True, [20000], [64], 2, 2, 128, 128),
    (False, [400, 120, 0, 800, 300, 64, 1, 511], [30, 12, 40, 7, 25, 32, 40, 1], 4, 3, 128, 32),
    (False, [400, 120, 0, 800, 300, 64, 1, 511], [30, 12, 32, 7, 25, 32, 32, 1], 8, 8, 64, 256),
    (False, [400, 120, 0, 800, 300, 64, 1, 511], [30, 12, 32, 7, 25, 32, 32, 1], 8, 3, 96, 16),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("what", ["plain", "cap and bias", "growing", "hidden"])
@pytest.mark.parametrize("cut,older,new,heads,group,D,page", TAKEN)
def test_the_wide_kernel(what, dt, cut, older, new, heads, group, D, page):
    c = ref.Cache(older, new, heads, D, page, seed=D + len(older), fill=0x7F)
    Hq = heads * group
    blocks, kw, ref_kw = _blocks(new, D, 5), {}, {}
    g = torch.Generator().manual_seed(3)
    if what == "cap and bias":
        slopes = torch.rand(Hq, generator=g) * 0.3
        depth = torch.cat([b.sum(-1) - 1 for b in blocks]).int()
        at = depth + torch.repeat_interleave(torch.tensor(older), torch.tensor(new)).int()
        ref_kw = dict(softcap=15.0, slopes=slopes, positions=at)
        kw = dict(softcap=15.0, slopes=slopes.cuda(), positions=at.cuda())
    if what == "growing":                            # and whole key tiles of no value, and of no weight
        for b in range(len(new)):
            n = -(-c.lens[b] // page)
            ids = c.table[b, :n].long()
            c.ks[ids] *= torch.exp2(torch.linspace(-4, 5, n))[:, None]
            c.vs[ids] *= torch.exp2(torch.rand(n, 1, generator=g) * 20 - 10)
            c.vs[ids[(torch.arange(n) * page // 128) % 2 == b % 2]] = 0
    if what == "hidden":
        blocks = [torch.rand(n, n, generator=g) < 0.2 for n in new]
        for b in range(len(new)):
            blocks[b][new[b] // 2] = False
            at = older[b] + new[b] - 1
            c.v.view(torch.uint8)[c.table[b, at // page], heads - 1, at % page, 9] = 0x7F
    q = _randn(D, c.T, Hq, D).to(DT[dt])
    space = ops.cache_tree_attention_workspace(c.T, Hq, *c.args())
    # (the split kernel's is a few MB, or none for contexts of at most 768 tokens)
    assert space > 2e7 if cut else space <= 1024 and c.table.shape[1] * page > 768
    out = _run(c, q.cuda(), blocks, **kw)
    _check(out, c, q, blocks, D ** -0.5, **ref_kw)
    assert torch.equal(out.nan_to_num(7.0), _run(c, q.cuda(), blocks, **kw).nan_to_num(7.0))
    if what == "plain":
        assert torch.equal(out, _run(c, -q.cuda(), blocks, scale=-D ** -0.5))


def test_long_context_and_wide_tree():
    for older, new, group, D in ([20011], [64], 4, 128), ([30001], [3], 2, 64), ([9000], [90], 2, 256):
        c = ref.Cache(older, new, 2, D, 128, seed=7, fill=0x7F)
        blocks = _blocks(new, 7, 12)
        q = _randn(9, c.T, 2 * group, D).half()
        out = _run(c, q.cuda(), blocks)
        _check(out, c, q, blocks, D ** -0.5)


def test_more_nodes_than_the_wide_kernel_takes():
    """700 and 1030 drafted tokens: masks of 17 words, on the kernel that splits along the context."""
    c = ref.Cache([1200, 3], [700, 1030], 1, 64, 64, seed=2, fill=0x7F)
    blocks = _blocks(c.new, 8, 40)
    q = _randn(4, c.T, 2, 64).half()
    out = _run(c, q.cuda(), blocks)
    _check(out, c, q, blocks, 0.125)


@pytest.mark.parametrize("new,D", [(3, 64), (40, 128), (5, 256)])
def test_past_32_bit_offsets(new, D):
    """Pages whose bytes, and scales, lie past 4 GB of their pools."""
    heads, page, older = 8, 256, 1300
    pages = 2 ** 32 // (heads * page * D) + 12
    c = ref.Cache([older], [new], heads, D, page, seed=3)
    used = c.table[0, : -(-c.lens[0] // page)].long()
    far = torch.arange(pages - len(used), pages).flip(0)
    kc = torch.zeros(pages, heads, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vc = torch.zeros_like(kc)
    ks, vs = torch.zeros(pages, heads, device="cuda"), torch.zeros(pages, heads, device="cuda")
    for small, large in ((c.k, kc), (c.v, vc), (c.ks, ks), (c.vs, vs)):
        raw = torch.uint8 if large is kc or large is vc else torch.float32
        large.view(raw)[far.cuda()] = small.view(raw)[used].cuda()
    table = far.to(torch.int32)[None].cuda()
    blocks = _blocks(c.new, 4)
    q = _randn(5, new, 2 * heads, D).half()
    out = ops.cache_tree_attention(q.cuda(), br.words(blocks).cuda(), kc, vc, ks, vs, table,
                                   torch.tensor(c.lens, dtype=torch.int32).cuda())
    _check(out, c, q, blocks, D ** -0.5)


def test_graph_and_stream():
    c = ref.Cache([1200, 90], [9, 30], 2, 128, 32, seed=9)
    blocks = _blocks(c.new, 9)
    q = _randn(1, c.T, 8, 128).half().cuda()
    masks, args = br.words(blocks).cuda(), c.args()
    want = ops.cache_tree_attention(q, masks, *args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = ops.cache_tree_attention(q, masks, *args, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.cache_tree_attention(q, masks, *args, out=out)
    q2 = _randn(2, c.T, 8, 128).half().cuda()
    q.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ops.cache_tree_attention(q2, masks, *args))


def test_index_errors_are_recorded():
    c = ref.Cache([100, 30], [4, 3], 2, 64, 16, seed=2)
    blocks = _blocks(c.new, 1)
    q = _randn(1, 7, 4, 64).half().cuda()
    masks = br.words(blocks).cuda()
    for what, change in ((2, lambda r: r[4].__setitem__((1, 0), 10 ** 6)),
                         (3, lambda r: r[5].__setitem__(1, 2)), (4, lambda r: r[6].__setitem__(2, 9))):
        args = c.args()
        change(args)
        ops.cache_tree_attention(q, masks, *args)
        st, info = ops.get_cache_error()
        assert st == 2 and info[2] == what, (what, st, info)


def test_refusals():
    c = ref.Cache([100, 30], [4, 3], 2, 64, 16, seed=2)
    q = torch.zeros(7, 4, 64, dtype=torch.float16, device="cuda")
    masks = torch.zeros(7, 1, dtype=torch.int64, device="cuda")
    args = c.args()
    for bad, error in ((masks.int(), TypeError), (masks[:6], ValueError), (masks.cpu(), ValueError),
                       (masks[:, 0], ValueError), (None, TypeError), (masks[:, :0], ValueError),
                       (masks.expand(7, 2)[:, ::2].t().contiguous().t(), None)):
        if error is None:
            ops.cache_tree_attention(q, bad, *args)
            continue
        with pytest.raises(error):
            ops.cache_tree_attention(q, bad, *args)
    with pytest.raises(ValueError, match="words"):
        ops.cache_tree_attention(torch.zeros(70, 4, 64, dtype=torch.float16, device="cuda"),
                                 torch.zeros(70, 1, dtype=torch.int64, device="cuda"), *args[:7], 70)
    for name, bad, error in (("positions", torch.zeros(6, dtype=torch.int32, device="cuda"), ValueError),
                             ("positions", torch.zeros(7, device="cuda"), TypeError),
                             ("slopes", torch.zeros(3, device="cuda"), ValueError),
                             ("out", torch.zeros(7, 4, 64, device="cuda"), TypeError)):
        with pytest.raises(error):
            ops.cache_tree_attention(q, masks, *args, **{name: bad})
    with pytest.raises(ops.B2BError, match="UNSUPPORTED"):
        ops.cache_tree_attention(q, masks, *args, out=q)
    assert ops.cache_tree_attention(q[:0], masks[:0], *args[:6]).shape == (0, 4, 64)
