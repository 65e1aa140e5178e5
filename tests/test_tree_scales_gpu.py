"""Attention of drafted trees whose references move within a key tile, and whose pages have scales that
are no numbers, against its 64-bit form."""
import math

import pytest
import torch

from gemm_conv_chains_gb300 import ops

import branch_ref as br
import decoder_ref as ref
from decoder_ref import TINY, UNIT

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}

# The wide kernel: contexts cut, units whole; of one row tile, whose key tiles two softmaxes share, and of two.
WIDE = [
    (True, [2600, 700], [60, 33], 8, 2, 128), (True, [2600, 900], [64, 20], 8, 4, 64),
    (True, [1800, 5, 0, 2000], [70, 128, 90, 1], 4, 3, 96), (True, [20000], [64], 2, 2, 128),
    (False, [400, 120, 0, 800, 300, 64, 1, 511], [30, 12, 40, 7, 25, 32, 40, 1], 4, 3, 128),
    (False, [400, 120, 0, 800, 300, 64, 1, 511], [30, 12, 32, 7, 25, 32, 32, 1], 8, 8, 64),
]
# The split kernel, whole and cut.
SPLIT = [([40, 300], [6, 20], 2, 1, 64), ([1200, 90], [9, 30], 2, 4, 128), ([700, 40], [14, 9], 2, 2, 256)]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ops.lib()
    ops.get_cache_error()
    yield
    st, info = ops.get_cache_error()
    assert st == 0, f"cache error word left set: {st} {info}"


def _trees(new, seed, spread=5):
    return [br.ancestors(br.tree(n, seed + b, spread)) for b, n in enumerate(new)]


def _queries(c, Hq, dt, seed):
    return torch.randn(c.T, Hq, c.D, generator=torch.Generator().manual_seed(seed)).to(DT[dt])


def _check(out, c, q, blocks, **kw):
    want, tol = br.tree_attention(c, q, blocks, c.D ** -0.5, **kw)
    tol = tol + UNIT[q.dtype] * (want.abs() + tol) + TINY[q.dtype]
    got = out.cpu().double()
    assert torch.equal(got.isnan(), want.isnan())
    bad = ~((got - want).abs() <= tol) & ~want.isnan()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[:3].tolist()}"


def _is_wide(c, Hq, cut):
    """(the split kernel's workspace is a few MB, or none for contexts of at most 768 tokens)"""
    space = ops.cache_tree_attention_workspace(c.T, Hq, *c.args())
    assert space > 2e7 if cut else space <= 1024 and c.table.shape[1] * c.page > 768


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("step", [6.0, 20.0, 40.0])
@pytest.mark.parametrize("cut,older,new,heads,group,D", WIDE)
def test_references_move_in_both_halves_of_a_key_tile(cut, older, new, heads, group, D, step, dt):
    """Scores that grow by 2^step from each 64 tokens to the next, on values that shrink with them: both
    halves of every key tile move the reference, and what the first half left, its probabilities and the
    output so far, is scaled for the second."""
    c = ref.Cache(older, new, heads, D, 64, seed=D + len(older), fill=0x7F)
    Hq = heads * group
    q = _queries(c, Hq, dt, 3) * 0.02
    q[..., 0] = 1.0
    # channel 0 alone carries the growth: code 1 beside smaller ones
    c.k.copy_((c.k.float() * 0.0005).to(c.k.dtype))
    c.k[..., 0] = 1.0
    size = math.log(2) * D ** 0.5
    for b, n in enumerate(c.lens):
        pages = -(-n // 64)
        ids = c.table[b, :pages].long()
        level = torch.arange(pages) % 24
        c.ks[ids] = (size * step * (level + 1.0))[:, None].expand(-1, heads)
        c.vs[ids] = torch.exp2(-(level % 12).float())[:, None] * 0.01
    blocks = _trees(c.new, D)
    _is_wide(c, Hq, cut)
    args = [q.cuda(), br.words(blocks).cuda(), *c.args()]
    out = ops.cache_tree_attention(*args)
    _check(out, c, q, blocks)
    assert torch.equal(out, ops.cache_tree_attention(*args))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("softcap", [0.0, 15.0])
@pytest.mark.parametrize("of", ["keys", "values"])
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("cut,older,new,heads,group,D", [(None, *s) for s in SPLIT] + WIDE)
def test_a_page_whose_scale_is_no_number(cut, older, new, heads, group, D, page, of, softcap, dt):
    """Pages of drafted tokens alone, a NaN as one head's scale: the rows that see any of their tokens are
    NaN, and those whose masks hide the whole page are not."""
    older = [n // page * page for n in older]
    c = ref.Cache(older, new, heads, D, page, seed=D + len(older), fill=0x7F)
    Hq = heads * group
    g = torch.Generator().manual_seed(11)
    blocks = [torch.rand(n, n, generator=g) < 0.3 for n in new]
    scales = c.ks if of == "keys" else c.vs
    for b, n in enumerate(new):
        at = page if n > page else 0                 # the second page of drafted tokens where there is one
        scales[c.table[b, (older[b] + at) // page], heads - 1] = math.nan
        mine = slice(at, min(at + page, n))
        blocks[b][0::3, mine] = False
        blocks[b][1::3, mine] = False                # and rows that see the page's last token only
        blocks[b][1::3, mine.stop - 1] = True
    if cut is not None:
        _is_wide(c, Hq, cut)
    q = _queries(c, Hq, dt, 5)
    out = ops.cache_tree_attention(q.cuda(), br.words(blocks).cuda(), *c.args(), softcap=softcap)
    _check(out, c, q, blocks, softcap=softcap)
    nan = out.isnan().cpu()
    assert not nan[:, : Hq - group].any() and bool((nan.all(-1) == nan.any(-1)).all())
    row = 0
    for n in new:
        assert not nan[row: row + n: 3].any()
        assert nan[row + 1: row + n: 3, Hq - group:].all()
        row += n
