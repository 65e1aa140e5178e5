"""The attention over the paged e4m3 cache where its numbers lie far apart, against 64 bits.
Allowed errors are each row's own: they follow from the keys that the row sees and from how much
it attends to them, so that a row of small values is held to small errors."""
import math

import pytest
import torch

from gemm_conv_chains_gb300 import ops

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


def _attention(c, q, scale, softcap=0.0):
    """(out, allowed error), float64 [T, q heads, D].  p the probabilities, s the page scales of the
    values, c their codes:
      scores       fp32 sums of D products in any order, and 16 roundings of the score itself, of its
                   exponent and of the scales' logarithms beside it (|log2 s| <= 64)
      P            fp16 of p s in a row's own unit, in which the largest p s that it sees is at least
                   1: half a step of 11 bits each, and 2^-25 of that largest below fp16's normal range
      the output   half a step of its type"""
    T, Hq, D = q.shape
    group = Hq // c.heads
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    at = 0
    for b, n in enumerate(c.new):
        length = c.lens[b]
        k, v = c.values(b, length)
        keys = torch.arange(length)
        vs = c.vs.double()[c.table[b, keys // c.page].long()]             # [length, heads]
        pos = torch.arange(length - n, length)
        seen = keys <= pos[:, None]
        for h in range(Hq):
            qh, kh, vh, sh = q[at: at + n, h].double(), k[h // group], v[h // group], vs[:, h // group]
            z = qh @ kh.T * scale
            size = qh.abs() @ kh.abs().T * abs(scale)
            delta = 2.0 ** -24 * ((D + 16) * size + 16 * (z.abs() + 64))
            if softcap:
                z = softcap * torch.tanh(z / softcap)                     # a factor of at most 1
                delta = delta + 2.0 ** -20 * z.abs()
            z = torch.where(seen, z, -math.inf)
            p = torch.softmax(z, -1)
            out[at: at + n, h] = p @ vh
            mag = torch.where(seen, p * (2.0 ** -11 + 2.0 ** -18 + 2 * delta), 0)
            code = torch.where(sh[:, None] > 0, vh.abs() / sh[:, None], 0)
            most = (p * sh).max(-1, keepdim=True).values
            tol[at: at + n, h] = mag @ vh.abs() + (p * delta).sum(-1, keepdim=True) * (p @ vh.abs()) \
                + 2.0 ** -25 * most * (seen.double() @ code)
        at += n
    return out, tol + UNIT[q.dtype] * (out.abs() + tol) + TINY[q.dtype]


def _check(got, c, q, scale, softcap=0.0):
    want, tol = _attention(c, q, scale, softcap)
    err = (got.cpu().double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}; worst {(err / tol).max()} of what is " \
                          f"allowed, first {bad.nonzero()[:3].tolist()}"


# ------------------------------------------------------------------------------------
# pages whose value scales lie far apart
# ------------------------------------------------------------------------------------

def _two_kinds(older, new, heads, D, page, drop, ahead, first, seed=0):
    """A cache whose every third page has a value scale of 1 and the others 2^-drop (`first`: the other
    way round), and whose keys give the small ones scores above the others' by `ahead` for
    queries of _ones."""
    c = ref.Cache(older, new, heads, D, page, seed=seed)
    c.ks[:] = 2.0 ** -6
    c.vs[:] = 1.0
    g = torch.Generator().manual_seed(seed + 1)
    for b, n in enumerate(c.lens):
        for j in range(-(-n // page)):
            small = (j % 3 != 0) != first
            pid = int(c.table[b, j])
            c.vs[pid] = 2.0 ** -drop if small else 1.0
            # code * 2^-6 * D (queries of 1) * scale D^-1/2: channels of one sign, and little noise
            level = (ahead if small else 0.0) * 64 / math.sqrt(D)
            code = level + 4 * torch.randn(heads, page, D, generator=g) / math.sqrt(D)
            c.k[pid] = code.to(ref.F8)
    return c


CASES = [([200], [1], 2, 4, 64, 16), ([1900], [1], 1, 4, 128, 16), ([300, 1000], [1, 1], 2, 8, 128, 64),
         ([150], [3], 2, 2, 256, 32), ([90, 60], [4, 5], 2, 4, 96, 16), ([900], [6], 1, 3, 192, 16),
         ([130, 7], [40, 30], 8, 4, 128, 16), ([60, 300], [150, 33], 8, 3, 64, 16),
         ([20, 100], [70, 40], 8, 4, 96, 32)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("drop,ahead", [(10, 4), (14, 8), (17, 10), (20, 6), (20, 14), (26, 18), (40, 24),
                                        (60, 50)])
@pytest.mark.parametrize("older,new,heads,group,D,page", CASES)
@pytest.mark.parametrize("first", [False, True])
def test_rows_that_attend_to_pages_of_small_scales(dt, drop, ahead, older, new, heads, group, D, page,
                                                   first):
    c = _two_kinds(older, new, heads, D, page, drop, ahead, first)
    # the outputs of the smallest scales stay well inside the output type's range
    c.vs *= 256.0 if dt == "f16" else 1.0
    q = torch.ones(c.T, heads * group, D) + 0.02 * _randn(D, c.T, heads * group, D)
    q = q.to(DT[dt])
    out = ops.cache_attention(q.cuda(), *c.args())
    _check(out, c, q, D ** -0.5)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("drop", [14, 20, 30])
def test_early_prompt_rows_do_not_feel_the_scales_of_later_tokens(dt, drop):
    """A prompt's first page has small values, the next ones, in the same tile of keys, large ones:
    the first 16 rows see the first page only."""
    c = ref.Cache([0] * 8, [40] * 8, 8, 128, 16, seed=6)
    for b in range(8):
        c.vs[c.table[b, 0].long()] = 0.02 * 2.0 ** -drop
    q = _randn(7, c.T, 16, 128).to(DT[dt])
    out = ops.cache_attention(q.cuda(), *c.args())
    _check(out, c, q, 128 ** -0.5)


@pytest.mark.parametrize("older,new,heads,group,D,page", CASES)
def test_value_scales_of_zero_and_of_nothing_appended(older, new, heads, group, D, page):
    """A page of zeros has the scale 2^-64; a scale of 0 stands for zeros too.  Both take weight."""
    c = ref.Cache(older, new, heads, D, page, seed=3)
    q = (_randn(D, c.T, heads * group, D) * 2).bfloat16()
    for b in range(len(new)):
        for j, s in ((0, 2.0 ** -64), (2, 0.0)):
            if c.table[b, j] >= 0:
                c.vs[c.table[b, j].long()] = s
    out = ops.cache_attention(q.cuda(), *c.args())
    _check(out, c, q, D ** -0.5)


# ------------------------------------------------------------------------------------
# pages past a row's reach
# ------------------------------------------------------------------------------------

@pytest.mark.parametrize("older,new,heads,group,D,page", [
    ([30], [8], 2, 1, 64, 16), ([14, 100], [5, 14], 1, 4, 128, 16), ([60], [8], 1, 2, 256, 16),
    ([0, 50] * 4, [40, 40] * 4, 8, 2, 128, 16), ([10, 0], [150, 200], 8, 4, 64, 32),
    ([100, 250], [64, 70], 8, 3, 96, 16)])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_a_page_that_a_row_does_not_reach_leaves_it_alone(older, new, heads, group, D, page, softcap):
    """The last page of each sequence: scales that are NaN or infinite, then a page number outside the
    pool.  Rows before it keep their bits, rows that see it do not stay finite."""
    c = ref.Cache(older, new, heads, D, page, seed=8)
    q = _randn(D, c.T, heads * group, D).half()
    want = ops.cache_attention(q.cuda(), *c.args(), softcap=softcap).cpu()
    pos = torch.cat([torch.arange(a, a + n) for a, n in zip(older, new)])
    last = torch.cat([torch.full((n,), (a + n - 1) // page * page) for a, n in zip(older, new)])
    before = pos < last
    assert before.any() and not before.all()
    pids = [int(c.table[b, (n - 1) // page]) for b, n in enumerate(c.lens)]
    for name, value in (("vs", math.nan), ("vs", math.inf), ("ks", math.nan), ("ks", math.inf)):
        keep = getattr(c, name).clone()
        getattr(c, name)[pids] = value
        got = ops.cache_attention(q.cuda(), *c.args(), softcap=softcap).cpu()
        setattr(c, name, keep)
        assert torch.equal(got[before], want[before]), (name, value)
        if name == "vs":
            assert not got[~before].isfinite().all(-1).any()
    args = c.args()
    for b, n in enumerate(c.lens):
        args[4][b, (n - 1) // page] = c.pages + 5
    got = ops.cache_attention(q.cuda(), *args, softcap=softcap).cpu()
    st, info = ops.get_cache_error()
    assert st == 2 and info[2] == 2
    assert torch.equal(got[before], want[before])


# ------------------------------------------------------------------------------------
# caps far above the scores, and far below
# ------------------------------------------------------------------------------------

CAPPED = [([700], [1], 2, 4, 64, 16), ([300, 20], [5, 3], 1, 4, 128, 32), ([100], [6], 1, 2, 256, 64),
          ([0, 200], [150, 70], 8, 4, 128, 16), ([30] * 6, [60] * 6, 8, 2, 64, 32)]


@pytest.mark.parametrize("softcap", [1e-40, 1e-3, 0.5, 50.0, 1e3, 1e4, 1e6, 1e30])
@pytest.mark.parametrize("older,new,heads,group,D,page", CAPPED)
def test_caps_from_tiny_to_huge(softcap, older, new, heads, group, D, page):
    c = ref.Cache(older, new, heads, D, page, seed=4)
    q = (_randn(D + 1, c.T, heads * group, D) * 6).half()
    q[0] = 0                                          # scores of zero
    out = ops.cache_attention(q.cuda(), *c.args(), softcap=softcap)
    _check(out, c, q, D ** -0.5, softcap)


# ------------------------------------------------------------------------------------
# query rows whose channels lie far apart
# ------------------------------------------------------------------------------------

@pytest.mark.parametrize("spread", [12, 18, 22, 27])
@pytest.mark.parametrize("older,new,heads,group,D,page", CAPPED)
def test_bf16_queries_with_channels_far_apart(spread, older, new, heads, group, D, page):
    """One channel is 2^spread times the others, and the keys have next to nothing in it."""
    c = ref.Cache(older, new, heads, D, page, seed=5)
    c.ks *= 2.0 ** (spread - 3)
    c.k[..., 3] = 0.0
    q = _randn(D + 2, c.T, heads * group, D) * 2.0 ** -spread
    q[..., 3] = _randn(D, c.T, heads * group).clamp(-2, 2)
    q = q.bfloat16()
    out = ops.cache_attention(q.cuda(), *c.args(), scale=8 * D ** -0.5)
    _check(out, c, q, 8 * D ** -0.5)


@pytest.mark.parametrize("exponent", [-130, -120, -60, 60, 112, 122])
@pytest.mark.parametrize("older,new,heads,group,D,page", [CAPPED[1], CAPPED[3]])
def test_bf16_queries_of_any_size(exponent, older, new, heads, group, D, page):
    c = ref.Cache(older, new, heads, D, page, seed=6)
    q = (_randn(D + 3, c.T, heads * group, D).double() * 2.0 ** exponent).bfloat16()
    scale = 2.0 ** (-exponent if exponent > -120 else 119)
    out = ops.cache_attention(q.cuda(), *c.args(), scale=scale * D ** -0.5)
    _check(out, c, q, float(torch.tensor(scale * D ** -0.5)), 0.0)
