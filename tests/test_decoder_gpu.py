"""Rotary positions, the append to the paged e4m3 cache and the attention over it, on the GPU
against their 64-bit forms.  Allowed errors follow from the roundings each operator states:
fp32 arithmetic, one rounding of an output, half an e4m3 step per code, fp16 probabilities."""
import math

import pytest
import torch

from gemm_conv_chains_gb300 import ops

import decoder_ref as ref
from decoder_ref import F8, TINY, UNIT

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


# ------------------------------------------------------------------------------------
# rotary
# ------------------------------------------------------------------------------------

def _check_rotary(got, x, cs, layout, inverse=False):
    want = ref.turn(x.double(), cs, layout, inverse)
    rot = 2 * cs.shape[1]
    mag = x.double().abs().amax() * 2
    tol = UNIT[x.dtype] * want.abs() + TINY[x.dtype] + 2.0 ** -22 * mag
    err = (got.cpu().double() - want).abs()
    assert (err <= tol).all(), (err - tol).max()
    assert torch.equal(got.cpu()[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 64, 64), (7, 3, 64, 32), (33, 40, 128, 128),
                                       (300, 5, 96, 48), (17, 2, 256, 64), (5, 9, 40, 16)])
def test_rotary(dt, layout, T, H, D, rot):
    x = _randn(T, T, H, D).to(DT[dt])
    table = ops.rotary_table(5000, rot)
    pos = torch.randint(5000, (T,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    cs = table.cpu().double()[pos.long()]
    y = ops.rotary(x.cuda(), table, pos.cuda(), layout)
    _check_rotary(y, x, cs, layout)
    back = ops.rotary(x.cuda(), table, pos.cuda(), layout, inverse=True)
    _check_rotary(back, x, cs, layout, inverse=True)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_strided_and_in_place(layout):
    T, H, D, rot = 19, 4, 64, 32
    rows = _randn(3, T, H + 3, D).to(torch.bfloat16).cuda()
    keep = rows.clone()
    x = rows[:, 1: 1 + H]
    table = ops.rotary_table(64, rot)
    pos = torch.arange(T, dtype=torch.int32).cuda()
    want = ops.rotary(x, table, pos, layout)
    assert ops.rotary(x, table, pos, layout, out=x).data_ptr() == x.data_ptr()
    assert torch.equal(x, want)
    assert torch.equal(rows[:, :1], keep[:, :1]) and torch.equal(rows[:, 1 + H:], keep[:, 1 + H:])


@pytest.mark.parametrize("dt,layout,T,H,D,rot,in_place", [
    ("f16", "half", 7501, 33, 64, 64, False), ("bf16", "interleaved", 5003, 20, 96, 96, True),
    ("bf16", "half", 30011, 7, 96, 48, True), ("f16", "half", 70001, 3, 48, 16, False),
    ("f16", "interleaved", 30001, 1, 256, 256, False), ("bf16", "interleaved", 4001, 1, 2048, 2048, False),
    ("bf16", "half", 2049, 130, 64, 64, True), ("f16", "interleaved", 9000, 11, 128, 64, True)])
def test_rotary_of_many_rows(dt, layout, T, H, D, rot, in_place):
    """Enough rows for the kernel that walks them; strided, and the same bits as short calls give."""
    rows = _randn(T, T, H + 1, D).to(DT[dt]).cuda()
    x = rows[:, :H]
    was = x.cpu()
    table = ops.rotary_table(2000, rot)
    pos = torch.randint(2000, (T,), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    cuda_pos = pos.cuda()
    pieces = [(a, min(a + 50, T)) for a in (0, T // 3, T - 50)]
    short = [ops.rotary(x[a:b], table, cuda_pos[a:b], layout) for a, b in pieces]
    beside = rows[:, H].clone()
    y = ops.rotary(x, table, cuda_pos, layout, out=x) if in_place else \
        ops.rotary(x, table, cuda_pos, layout)
    assert torch.equal(rows[:, H], beside)
    for (a, b), want in zip(pieces, short):
        assert torch.equal(y[a:b], want)
    _check_rotary(y, was, table.cpu().double()[pos.long()], layout)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_gradient_is_the_inverse(layout):
    """<rotary(x), w> differentiated: by the formula (the inverse of w) and by differences."""
    T, H, D, rot = 6, 2, 64, 48
    x, w = _randn(5, T, H, D).half(), _randn(6, T, H, D).half()
    table = ops.rotary_table(900, rot)
    pos = torch.arange(T, dtype=torch.int32) * 131
    grad = ops.rotary(w.cuda(), table, pos.cuda(), layout, inverse=True).cpu().double()
    cs = table.cpu().double()[pos.long()]
    xx = x.double().requires_grad_(True)
    (ref.turn(xx, cs, layout) * w.double()).sum().backward()
    tol = UNIT[torch.float16] * xx.grad.abs() + 2.0 ** -22 * 8 + TINY[torch.float16]
    assert ((grad - xx.grad).abs() <= tol).all()
    # the rotation is linear: a step of 1 in one channel changes the sum by its gradient; the
    # two outputs of its pair are each rounded twice (fp16, |y| < 8: 2^-9 each way)
    base = ops.rotary(x.cuda(), table, pos.cuda(), layout).cpu().double()
    for t, h, d in [(0, 0, 0), (3, 1, 17), (5, 0, 47), (4, 1, 60)]:
        moved = x.clone()
        moved[t, h, d] = 0 if x[t, h, d].abs() > 1 else x[t, h, d] + 1
        step = (moved[t, h, d].double() - x[t, h, d].double()).item()
        y = ops.rotary(moved.cuda(), table, pos.cuda(), layout).cpu().double()
        diff = ((y - base) * w.double()).sum().item() / step
        room = 4 * 2.0 ** -9 * w.abs().max().item() / abs(step)
        assert abs(diff - grad[t, h, d].item()) <= room + 2.0 ** -9


def test_rotary_table_scalings():
    n, rot = 70000, 64
    plain = ops.rotary_table(n, rot, base=500000.0).cpu().double()
    want = ref.table64(n, rot, 500000.0)
    # fp64 angle (|angle| < 7e4: its rounding is below 1e-11), one rounding to fp32
    assert ((plain - want).abs() <= 2.0 ** -24 + 1e-10).all()
    line = ops.rotary_table(n, rot, scaling="linear", factor=4.0).cpu().double()
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    pos = torch.arange(n, dtype=torch.float64)[:, None]
    f = 10000.0 ** (-i / rot)
    assert ((line[..., 0] - (pos * (f / 4)).cos()).abs() <= 2.0 ** -24 + 1e-10).all()
    blend = ops.rotary_table(n, rot, scaling="blend", factor=8.0, original=4096, low=1.0, high=32.0,
                             gain=1.25).cpu().double()
    keep = ((4096 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
    a = pos * (keep * f + (1 - keep) * f / 8.0)
    want = torch.stack([a.cos(), a.sin()], -1) * 1.25
    assert ((blend - want).abs() <= 1.25 * 2.0 ** -24 + 1e-9).all()


def test_rotary_position_outside_the_table_is_recorded():
    x = torch.ones(3, 2, 64, dtype=torch.float16).cuda()
    table = ops.rotary_table(10, 64)
    out = torch.full_like(x, 7)
    ops.rotary(x, table, torch.tensor([0, 10, -1], dtype=torch.int32).cuda(), out=out)
    st, info = ops.get_cache_error()
    assert st == 2 and info[2] == 1 and info[3] in (1, 2)
    assert torch.equal(out[0], x[0]) and (out[1:] == 7).all()


# ------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------

def _half_step(y):
    """Half an e4m3 step around y (|y| <= 448), float64."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6)))
    return torch.exp2(e - 4)


def _check_append(c, codes, scale, was, was_scale, new):
    """codes, scale after the append against the definition; new [T, heads, D] float64."""
    touched = torch.zeros(c.pages, c.page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(c.new):
        a = c.older[b]
        if n == 0:
            continue
        for j in range(a // c.page, (a + n - 1) // c.page + 1):
            lo, hi = max(a, j * c.page), min(a + n, (j + 1) * c.page)
            pid, held = int(c.table[b, j]), max(0, a - j * c.page)
            part = new[at + lo - a: at + hi - a].transpose(0, 1)
            top = torch.where(part.isfinite(), part.abs(), 0).amax((1, 2))
            s0 = was_scale[pid].double() if held else torch.zeros(c.heads, dtype=torch.float64)
            s1 = torch.maximum(s0, top / 448).clamp_min(2.0 ** -64)
            got_s = scale[pid].double()
            assert ((got_s - s1).abs() <= 2.0 ** -22 * s1).all()
            got = codes[pid].double()
            want = (part / got_s[:, None, None]).clamp(-448, 448)
            mine = got[:, lo - j * c.page: hi - j * c.page]
            assert torch.equal(mine.isnan(), want.isnan())
            ok = (mine - want).abs() <= _half_step(want) * (1 + 2.0 ** -18) + 2.0 ** -30
            assert (ok | want.isnan()).all()
            old = was[pid].double()[:, :held]
            moved = old * (s0 / got_s)[:, None, None]
            grew = (got_s > s0)[:, None, None]
            assert torch.equal(torch.where(grew, 0.0, got[:, :held]), torch.where(grew, 0.0, old))
            assert ((got[:, :held] - moved).abs() <=
                    torch.where(grew, _half_step(moved) * (1 + 2.0 ** -18), 0.0)).all()
            touched[pid, : hi - j * c.page] = True
        at += n
    same = codes.view(torch.uint8) == was.view(torch.uint8)
    assert same.transpose(1, 2)[~touched].all()
    lone = ~touched.any(1)
    assert torch.equal(scale[lone], was_scale[lone])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("older,new,heads,D,rot,page", [
    ([0], [1], 1, 64, 64, 16), ([5, 16, 31, 0], [1, 1, 1, 1], 2, 128, 64, 16),
    ([0, 17, 64, 200], [50, 1, 0, 131], 3, 64, 32, 64), ([3], [700], 2, 96, 96, 256),
    ([127, 128], [1, 2], 5, 256, 128, 128), ([9, 40], [33, 64], 4, 192, 192, 32)])
def test_append(dt, layout, older, new, heads, D, rot, page):
    c = ref.Cache(older, new, heads, D, page, seed=len(older))
    rows = _randn(D + page, c.T, 3 * heads + 2, D).to(DT[dt])
    rows[:, heads:2 * heads] *= 3
    k, v, q = rows[:, :heads], rows[:, heads:2 * heads], rows[:, 2 * heads:]
    dev = rows.cuda()
    table = ops.rotary_table(max(c.lens), rot)
    kc, vc, ks, vs, *rest = c.args()
    q_out = ops.cache_append(dev[:, :heads], dev[:, heads:2 * heads], kc, vc, ks, vs, *rest,
                             table=table, layout=layout, q=dev[:, 2 * heads:])
    pos = torch.cat([torch.arange(a, a + n) for a, n in zip(older, new)])
    cs = table.cpu().double()[pos]
    _check_append(c, kc.cpu(), ks.cpu(), c.k, c.ks, ref.turn(k.double(), cs, layout))
    _check_append(c, vc.cpu(), vs.cpu(), c.v, c.vs, v.double())
    _check_rotary(q_out, q, cs, layout)
    again = [t.clone() for t in (kc, vc, ks, vs)]
    ops.cache_append(dev[:, :heads], dev[:, heads:2 * heads], kc, vc, ks, vs, *rest, table=table,
                     layout=layout)
    for x, y in zip(again, (kc, vc, ks, vs)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_append_turns_the_queries_of_many_rows(layout):
    """Enough query rows for the kernel that walks them, over ragged and empty sequences."""
    older, new, heads, D, q_heads = [5, 0, 100, 3, 0], [1500, 0, 2111, 1, 700], 1, 64, 61
    c = ref.Cache(older, new, heads, D, 32, seed=9)
    rows = _randn(D, c.T, 2 * heads + q_heads, D).to(torch.bfloat16)
    dev = rows.cuda()
    table = ops.rotary_table(max(c.lens), D)
    kc, vc, ks, vs, *rest = c.args()
    q = dev[:, 2 * heads:]
    q_out = ops.cache_append(dev[:, :heads], dev[:, heads:2 * heads], kc, vc, ks, vs, *rest,
                             table=table, layout=layout, q=q)
    pos = torch.cat([torch.arange(a, a + n) for a, n in zip(older, new)]).int()
    _check_rotary(q_out, rows[:, 2 * heads:], table.cpu().double()[pos.long()], layout)
    assert torch.equal(q_out[1400:1600], ops.rotary(q[1400:1600], table, pos[1400:1600].cuda(), layout))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_append_sends_exact_ties_to_even(dt):
    """Values of few bits: y * 448 / A often lies exactly between two codes.  The quotient of such
    short numbers is never close to a tie without being one, so the codes have one right answer."""
    c = ref.Cache([0, 0], [64, 70], 2, 64, 32, seed=5)
    v = (_randn(21, c.T, 2, 64) * 37).round().clamp(-112, 112).to(DT[dt])
    v[:64, 0] *= 2 ** -5
    v[3, 1, 7] = 126                                  # pages whose A is not a power of two times 7
    v[90, 0, 1] = -121
    kc, vc, ks, vs, *rest = c.args()
    ops.cache_append(torch.zeros_like(v).cuda(), v.cuda(), kc, vc, ks, vs, *rest)
    vc = vc.cpu()
    ties = 0
    for b, (at, n) in enumerate([(0, 64), (64, 70)]):
        for j in range(-(-n // 32)):
            part = v[at + 32 * j: at + min(n, 32 * j + 32)].double().transpose(0, 1)
            A = part.abs().amax((1, 2), keepdim=True)
            x = part * 448 / A
            want = x.float().to(F8)
            got = vc[c.table[b, j], :, : part.shape[1]]
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
            down = (x.float() * (1 - 2.0 ** -20)).to(F8).float()
            up = (x.float() * (1 + 2.0 ** -20)).to(F8).float()
            ties += int((down != up).sum())
    assert ties > 100


def test_append_without_rotation_or_starts():
    c = ref.Cache([30, 0, 5], [2, 2, 2], 2, 64, 16, seed=2)
    k, v = _randn(1, 6, 2, 64).half(), _randn(2, 6, 2, 64).half() * 0.001
    kc, vc, ks, vs, *rest = c.args(starts=False)
    assert ops.cache_append(k.cuda(), v.cuda(), kc, vc, ks, vs, *rest) is None
    _check_append(c, kc.cpu(), ks.cpu(), c.k, c.ks, k.double())
    _check_append(c, vc.cpu(), vs.cpu(), c.v, c.vs, v.double())


def test_append_zeros_infinities_and_nans():
    c = ref.Cache([0, 20], [3, 3], 2, 64, 16, seed=4)
    k, v = _randn(1, 6, 2, 64).bfloat16(), torch.zeros(6, 2, 64).bfloat16()
    k[0, 0, 3], k[1, 1, 5], k[4, 0, 63], v[5, 1, 0] = math.inf, math.nan, -math.inf, math.nan
    kc, vc, ks, vs, *rest = c.args()
    ops.cache_append(k.cuda(), v.cuda(), kc, vc, ks, vs, *rest)
    _check_append(c, kc.cpu(), ks.cpu(), c.k, c.ks, k.double())
    _check_append(c, vc.cpu(), vs.cpu(), c.v, c.vs, v.double())
    assert vs.cpu()[c.table[0, 0]].eq(2.0 ** -64).all()


def test_append_token_by_token_stays_within_the_steps_of_each_growth():
    """Tokens that arrive one by one, each larger than the last: every append re-quantises the
    page, and each time adds at most half a step."""
    D, page, n = 64, 16, 16
    x = _randn(8, n, 1, D).half()
    x *= torch.linspace(0.5, 4, n)[:, None, None].half()
    c = ref.Cache([0], [n], 1, D, page, spare=0)
    kc, vc, ks, vs, table, *_ = c.args()
    for i in range(n):
        lens = torch.tensor([i + 1], dtype=torch.int32).cuda()
        ops.cache_append(x[i: i + 1].cuda(), x[i: i + 1].cuda(), kc, vc, ks, vs, table, lens)
    got = kc.cpu()[0, 0].double() * ks.cpu()[0, 0].double()
    want = x[:, 0].double()
    room = torch.zeros_like(want)
    for i in range(n):                                # s at most the final one at every step
        room[:i + 1] += torch.maximum(want[:i + 1].abs() * 2.0 ** -4, ks.cpu()[0, 0] * 2.0 ** -10)
    assert ((got - want).abs() <= room).all()
    assert torch.equal(kc.view(torch.uint8), vc.view(torch.uint8))


def test_append_index_errors_are_recorded_and_write_nothing():
    c = ref.Cache([0, 4], [2, 2], 1, 64, 16, seed=1)
    k = _randn(1, 4, 1, 64).half().cuda()
    for what, change in [(2, lambda r: r[0].__setitem__((1, 0), c.pages)),
                         (2, lambda r: r[0].__setitem__((1, 0), -1)),
                         (3, lambda r: r[1].__setitem__(1, 1)),
                         (3, lambda r: r[1].__setitem__(1, 1000)),
                         (4, lambda r: r[2].__setitem__(2, 9)),
                         (4, lambda r: r[2].__setitem__(2, 1))]:
        kc, vc, ks, vs, *rest = c.args()
        change(rest)
        before = kc.clone()
        ops.cache_append(k, k, kc, vc, ks, vs, *rest)
        st, info = ops.get_cache_error()
        assert st == 2 and info[2] == what and info[3] == 1, (what, info)
        own = int(c.table[0, 0])
        others = [i for i in range(c.pages) if i != own]
        assert torch.equal(kc.view(torch.uint8)[others], before.view(torch.uint8)[others])
    table = ops.rotary_table(5, 64)
    kc, vc, ks, vs, *rest = c.args()
    ops.cache_append(k, k, kc, vc, ks, vs, *rest, table=table)
    st, info = ops.get_cache_error()
    assert st == 2 and info[2] == 1 and info[3] == 1


# ------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------

def _check_attention(got, c, q, scale, softcap=0.0, slopes=None):
    want, tol = ref.attention(c, q, scale, softcap, slopes)
    tol = tol + UNIT[q.dtype] * (want.abs() + tol) + TINY[q.dtype]
    got = got.cpu().double()
    assert torch.equal(got.isnan(), want.isnan()) or not want.isnan().any() and not got.isnan().any()
    err = (got - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}; worst {(err - tol).max()}, " \
                          f"first {bad.nonzero()[:3].tolist()}"


SHAPES = [
    ([0], [1], 1, 1, 64, 16), ([199], [1], 4, 1, 64, 16), ([15, 16, 17, 255], [1] * 4, 2, 4, 128, 16),
    ([1000, 3, 513, 64], [1] * 4, 2, 8, 128, 64), ([700, 0, 40], [1] * 3, 1, 16, 128, 32),
    ([300, 2], [1, 1], 2, 5, 96, 32), ([77, 511], [1, 1], 2, 3, 192, 128),
    ([530, 1040], [1, 1], 1, 8, 256, 256), ([100, 7, 0], [4, 3, 5], 2, 2, 64, 64),
    ([600, 31], [7, 2], 2, 4, 256, 32), ([90, 1100], [40, 9], 1, 5, 128, 16),
    ([0, 33], [150, 70], 2, 2, 64, 32), ([0], [130], 1, 3, 96, 16), ([64], [65], 2, 4, 128, 64),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("older,new,heads,group,D,page", SHAPES)
def test_attention(dt, older, new, heads, group, D, page):
    """Every head size, row tile and split; whatever no token was written to is NaN."""
    c = ref.Cache(older, new, heads, D, page, seed=D + len(older), fill=0x7F)
    Hq = heads * group
    rows = _randn(D, c.T, Hq + 2, D).to(DT[dt])
    out = ops.cache_attention(rows.cuda()[:, 1: 1 + Hq], *c.args())
    _check_attention(out, c, rows[:, 1: 1 + Hq], D ** -0.5)


# Enough rows and heads for the kernel that takes prompts (256 query rows per block): ragged, rows
# that end inside a row tile, contexts that end inside a key tile, sequences with one new token.
PROMPTS = [
    ([0, 100, 7, 300, 64, 1, 130, 255], [70, 1, 33, 40, 64, 2, 65, 10], 8, 2, 64, 16),
    ([0, 900, 250, 3], [150, 129, 1, 260], 8, 3, 128, 32),
    ([1000, 40], [300, 257], 8, 4, 128, 64), ([5, 0, 700], [100, 200, 64], 8, 4, 96, 128),
    ([129, 0, 17, 511], [128, 1, 90, 65], 16, 1, 64, 256), ([0], [1100], 4, 2, 128, 16),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("older,new,heads,group,D,page", PROMPTS)
def test_attention_of_prompts(dt, older, new, heads, group, D, page):
    c = ref.Cache(older, new, heads, D, page, seed=D + len(older), fill=0xFF)
    Hq = heads * group
    rows = _randn(D, c.T, Hq + 1, D).to(DT[dt])
    out = ops.cache_attention(rows.cuda()[:, :Hq], *c.args())
    _check_attention(out, c, rows[:, :Hq], D ** -0.5)
    assert torch.equal(out, ops.cache_attention(rows.cuda()[:, :Hq], *c.args()))
    back = ops.cache_attention(-rows.cuda()[:, :Hq], *c.args(), scale=-D ** -0.5)
    assert torch.equal(out, back)


def _prompt_case(seed, new=40):
    return ref.Cache([50 + 9 * i for i in range(8)], [new] * 8, 8, 128, 32, seed=seed)


def test_prompt_scores_and_scales_far_apart():
    c = _prompt_case(3)
    c.ks *= torch.exp2(torch.linspace(-3, 6, c.pages))[:, None]
    c.vs *= torch.exp2(torch.linspace(8, -12, c.pages))[:, None]
    c.vs[5] = 0
    q = (_randn(2, c.T, 16, 128) * 3).bfloat16()
    out = ops.cache_attention(q.cuda(), *c.args())
    _check_attention(out, c, q, 128 ** -0.5)


def test_prompt_infinite_and_nan_inputs_stay_in_their_rows():
    c = _prompt_case(4)
    q = _randn(3, c.T, 16, 128).half()
    want = ops.cache_attention(q.cuda(), *c.args()).cpu()
    rows = torch.ones(c.T, 16, 128, dtype=torch.bool)
    at = 3 * 40                                        # the fourth sequence
    q[at + 2, 1, 7], q[at + 3, 0, 0] = math.nan, math.inf
    rows[at + 2, 1] = rows[at + 3, 0] = False
    place = c.older[3] + 20                            # its 21st new token: a value and a key
    pid, slot = int(c.table[3, place // 32]), place % 32
    c.v[pid, 2, slot, 9] = math.nan                    # query heads 4 and 5
    c.k[pid, 6, slot, 100] = math.nan                  # query heads 12 and 13
    rows[at + 20: at + 40, 4:6, 9] = False
    rows[at + 20: at + 40, 12:14] = False
    got = ops.cache_attention(q.cuda(), *c.args()).cpu()
    assert torch.equal(got[rows], want[rows])
    assert got[~rows].isnan().all()


def test_prompt_index_errors_are_recorded():
    c = _prompt_case(5)
    q = _randn(5, c.T, 16, 128).half().cuda()
    want = ops.cache_attention(q, *c.args())
    for what, change in [(2, lambda r: r[4].__setitem__((2, 1), c.pages)),
                         (2, lambda r: r[4].__setitem__((2, 0), -7)),
                         (3, lambda r: r[5].__setitem__(2, 39)),
                         (3, lambda r: r[5].__setitem__(2, 10 ** 6)),
                         (4, lambda r: r[6].__setitem__(8, 400))]:
        args = c.args()
        change(args)
        got = ops.cache_attention(q, *args)
        st, info = ops.get_cache_error()
        assert st == 2 and info[2] == what and info[3] == (7 if what == 4 else 2), (what, info)
        assert torch.equal(got[:80], want[:80]) and torch.equal(got[120:280], want[120:280])


@pytest.mark.parametrize("softcap,bias", [(20.0, False), (0.0, True), (5.0, True)])
@pytest.mark.parametrize("older,new,heads,group,D,page", [SHAPES[3], SHAPES[9], SHAPES[11], PROMPTS[0],
                                                          PROMPTS[1], PROMPTS[3]])
def test_attention_cap_and_bias(softcap, bias, older, new, heads, group, D, page):
    c = ref.Cache(older, new, heads, D, page, seed=7, fill=0xFF)
    Hq = heads * group
    q = (_randn(D, c.T, Hq, D) * 3).bfloat16()
    slopes = torch.exp2(-torch.arange(1.0, Hq + 1)) if bias else None
    out = ops.cache_attention(q.cuda(), *c.args(), scale=0.2, softcap=softcap,
                              slopes=None if slopes is None else slopes.cuda())
    _check_attention(out, c, q, 0.2, softcap, slopes)


def test_attention_even_rows_without_starts_and_a_given_workspace():
    c = ref.Cache([900, 1500, 2], [2, 2, 2], 2, 64, 32, seed=9)
    q = _randn(4, 6, 8, 64).half()
    args = c.args(starts=False)
    need = ops.cache_attention_workspace(6, 8, *args)
    assert need > 0
    work = torch.full((need,), 0xFF, dtype=torch.uint8).cuda()
    out = torch.full((6, 8, 64), 5.0, dtype=torch.float16).cuda()
    assert ops.cache_attention(q.cuda(), *args, out=out, workspace=work) is out
    _check_attention(out, c, q, 64 ** -0.5)
    assert torch.equal(out, ops.cache_attention(q.cuda(), *args))      # no order left to chance


def test_attention_huge_and_tiny_scales_of_pages():
    """Value scales over many powers of two within one sequence, dominant keys among them."""
    c = ref.Cache([1500], [1], 1, 128, 16, seed=12)
    c.vs *= torch.exp2(torch.linspace(-30, 10, c.pages))[:, None]
    q = _randn(1, 1, 4, 128).half()
    out = ops.cache_attention(q.cuda(), *c.args())
    _check_attention(out, c, q, 128 ** -0.5)
    c.vs[:] = 0                                       # values of nothing are zero
    assert not ops.cache_attention(q.cuda(), *c.args()).any()


def test_attention_large_scores():
    """Scores far apart: the maximum moves by more than the reference's slack many times."""
    c = ref.Cache([1200], [1], 1, 64, 16, seed=13)
    c.ks *= torch.linspace(0.1, 40, c.pages)[:, None]
    q = (_randn(2, 1, 8, 64) * 4).bfloat16()
    out = ops.cache_attention(q.cuda(), *c.args())
    _check_attention(out, c, q, 64 ** -0.5)


def test_attention_infinite_and_nan_inputs_stay_in_their_rows():
    c = ref.Cache([50], [5], 1, 64, 64, seed=14)
    q = _randn(3, 5, 2, 64).half()
    q[2, 1, 7] = math.nan
    q[3, 0, 0] = math.inf
    pid = int(c.table[0, 0])
    c.v[pid, 0, 53, 9] = math.nan                     # the fourth new token's value
    got = ops.cache_attention(q.cuda(), *c.args()).cpu()
    assert got[2, 1].isnan().all() and got[3, 0].isnan().all()
    assert got[3:, :, 9].isnan().all()
    clean = ref.Cache([50], [5], 1, 64, 64, seed=14)
    want = ops.cache_attention(_randn(3, 5, 2, 64).half().cuda(), *clean.args()).cpu()
    rows = torch.ones(5, 2, 64, dtype=torch.bool)
    rows[2, 1] = rows[3, 0] = False
    rows[3:, :, 9] = False
    assert torch.equal(got[rows], want[rows])


def test_attention_on_another_stream():
    c = ref.Cache([3000, 10], [1, 1], 2, 128, 64, seed=15)
    q = _randn(3, 2, 8, 128).bfloat16()
    args, qd = c.args(), q.cuda()
    want = ops.cache_attention(qd, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.cache_attention(qd, *args, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_attention_past_32_bit_offsets():
    """A pool of more than 2^32 bytes, the sequence's pages at its end."""
    heads, page, D = 8, 64, 128
    pages = 2 ** 32 // (heads * page * D) + 40
    small = ref.Cache([130, 700], [1, 1], heads, D, page, seed=16)
    q = _randn(5, 2, 8, 128).half()
    kc = torch.empty(pages, heads, page, D, dtype=F8, device="cuda")
    vc = torch.empty_like(kc)
    ks = torch.empty(pages, heads, device="cuda")
    vs = torch.empty_like(ks)
    shift = pages - small.pages
    kc[shift:], vc[shift:] = small.k.cuda(), small.v.cuda()
    ks[shift:], vs[shift:] = small.ks.cuda(), small.vs.cuda()
    args = small.args()
    table = torch.where(args[4] >= 0, args[4] + shift, -1).to(torch.int32)
    got = ops.cache_attention(q.cuda(), kc, vc, ks, vs, table, *args[5:])
    assert torch.equal(got, ops.cache_attention(q.cuda(), *args))
    k = _randn(6, 2, heads, D).half().cuda()
    ops.cache_append(k, k, kc, vc, ks, vs, table, *args[5:])
    ops.cache_append(k, k, *args)
    assert torch.equal(kc[shift:].view(torch.uint8), args[0].view(torch.uint8))
    assert torch.equal(ks[shift:], args[2])


def test_prompts_past_32_bit_offsets():
    """The same for prompts, with query rows that lie 2^24 elements apart."""
    heads, page, D, Hq = 8, 32, 128, 16
    pages = 2 ** 32 // (heads * page * D) + 200
    small = _prompt_case(17, new=40)
    q = _randn(8, small.T, Hq, D).half().cuda()
    far = torch.empty(small.T * 2 ** 24, dtype=torch.float16, device="cuda").as_strided(
        (small.T, Hq, D), (2 ** 24, D, 1))
    far.copy_(q)
    kc = torch.empty(pages, heads, page, D, dtype=F8, device="cuda")
    vc = torch.empty_like(kc)
    ks = torch.empty(pages, heads, device="cuda")
    vs = torch.empty_like(ks)
    shift = pages - small.pages
    kc[shift:], vc[shift:] = small.k.cuda(), small.v.cuda()
    ks[shift:], vs[shift:] = small.ks.cuda(), small.vs.cuda()
    args = small.args()
    table = torch.where(args[4] >= 0, args[4] + shift, -1).to(torch.int32)
    got = ops.cache_attention(far, kc, vc, ks, vs, table, *args[5:])
    assert torch.equal(got, ops.cache_attention(q, *args))


@pytest.mark.parametrize("T", [260, 9000])
def test_rotary_past_32_bit_offsets(T):
    """Rows far apart, few of them and enough for the kernel that walks them."""
    H, D = 20, 64
    ld = 2 ** 33 // T // 8 * 8
    x = _randn(T, T, H, D).bfloat16().cuda()
    far = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").as_strided((T, H, D), (ld, D, 1))
    far.copy_(x)
    table = ops.rotary_table(100, D)
    pos = (torch.arange(T, dtype=torch.int32) % 100).cuda()
    want = ops.rotary(x, table, pos, "interleaved")
    assert torch.equal(ops.rotary(far, table, pos, "interleaved", out=far), want)


def test_attention_index_errors_are_recorded():
    c = ref.Cache([100, 40], [1, 1], 2, 64, 16, seed=17)
    q = _randn(5, 2, 4, 64).half().cuda()
    want = ops.cache_attention(q, *c.args())
    for what, change in [(2, lambda r: r[4].__setitem__((1, 1), c.pages)),
                         (2, lambda r: r[4].__setitem__((1, 1), -7)),
                         (3, lambda r: r[5].__setitem__(1, 0)),
                         (3, lambda r: r[5].__setitem__(1, 10 ** 6)),
                         (4, lambda r: r[6].__setitem__(2, 3))]:
        args = c.args()
        change(args)
        got = ops.cache_attention(q, *args)
        st, info = ops.get_cache_error()
        assert st == 2 and info[2] == what and info[3] == 1, (what, info)
        assert torch.equal(got[0], want[0])


def test_no_rows_is_no_launch():
    c = ref.Cache([5], [1], 1, 64, 16)
    args = c.args(starts=False)
    q = torch.empty(0, 2, 64, dtype=torch.float16).cuda()
    assert ops.cache_attention(q, *args).shape == (0, 2, 64)
    k = torch.empty(0, 1, 64, dtype=torch.float16).cuda()
    before = args[0].clone()
    ops.cache_append(k, k, *args)
    assert torch.equal(before.view(torch.uint8), args[0].view(torch.uint8))
    table = ops.rotary_table(4, 64)
    assert ops.rotary(q, table, torch.empty(0, dtype=torch.int32).cuda()).shape == (0, 2, 64)


# ------------------------------------------------------------------------------------
# refusals of the binding that need CUDA tensors
# ------------------------------------------------------------------------------------

def test_binding_refuses_wrong_operands():
    c = ref.Cache([5, 7], [1, 1], 2, 64, 16)
    args = c.args(starts=False)
    q = torch.zeros(2, 4, 64, dtype=torch.float16, device="cuda")
    k = torch.zeros(2, 2, 64, dtype=torch.float16, device="cuda")

    def other(i, t):
        return args[:i] + [t] + args[i + 1:]

    for i, t, error in [(0, args[0].view(torch.uint8), TypeError), (1, args[1][:1], ValueError),
                        (0, args[0].transpose(1, 2), ValueError), (2, args[2].double(), TypeError),
                        (2, args[2].cpu(), ValueError), (3, args[3][:, :1], ValueError),
                        (4, args[4].long(), TypeError), (4, args[4][0], ValueError),
                        (5, args[5][:1], ValueError), (5, args[5].cpu(), ValueError)]:
        with pytest.raises(error):
            ops.cache_attention(q, *other(i, t))
        with pytest.raises(error):
            ops.cache_append(k, k, *other(i, t))
    with pytest.raises(ValueError, match="starts has shape"):
        ops.cache_attention(q, *args, starts=args[5])
    with pytest.raises(ValueError, match="head size"):
        ops.cache_attention(torch.zeros(2, 4, 128, dtype=torch.float16, device="cuda"), *args)
    with pytest.raises(ValueError, match="dense heads"):
        ops.cache_attention(q.transpose(0, 1).contiguous().transpose(0, 1), *args)
    with pytest.raises(TypeError, match="out has dtype"):
        ops.cache_attention(q, *args, out=q.float())
    with pytest.raises(TypeError, match="slopes has dtype"):
        ops.cache_attention(q, *args, slopes=torch.zeros(4, dtype=torch.float16, device="cuda"))
    with pytest.raises(ops.B2BError):                        # 3 query heads over 2 kv heads
        ops.cache_attention(q[:, :3], *args)
    with pytest.raises(ops.B2BError):
        ops.cache_attention(q, *args, softcap=-1.0)
    with pytest.raises(ValueError, match="needs a table"):
        ops.cache_append(k, k, *args, q=q)
    with pytest.raises(ValueError, match="without q"):
        ops.cache_append(k, k, *args, q_out=q)
    with pytest.raises(TypeError, match="v has dtype"):
        ops.cache_append(k, k.bfloat16(), *args)
    table = ops.rotary_table(20, 64)
    with pytest.raises(ValueError, match="table has shape"):
        ops.rotary(q, table[..., 0], args[5])
    with pytest.raises(TypeError, match="positions has dtype"):
        ops.rotary(q, table, args[5].long())
    with pytest.raises(ops.B2BError):                        # rot above the head's channels
        ops.rotary(q, ops.rotary_table(20, 128), args[5])
    long = ref.Cache([4000], [1], 1, 64, 16)
    with pytest.raises(ops.B2BError):
        ops.cache_attention(q[:1], *long.args(starts=False),
                            workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_streams_by_object_and_handle():
    x = _randn(1, 9, 3, 64).half().cuda()
    table = ops.rotary_table(50, 64)
    pos = torch.arange(9, dtype=torch.int32).cuda()
    want = ops.rotary(x, table, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    by_object = ops.rotary(x, table, pos, stream=side)
    by_handle = ops.rotary(x, table, pos, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(by_object, want) and torch.equal(by_handle, want)
