"""The decoder-block operators at batch sizes past each kernel's first stretch of sequences, with long
prompts at wide heads, captured into graphs, and from several streams and threads at once."""
import copy
import random
import threading

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


def _check(got, c, q, scale, softcap=0.0):
    c = copy.copy(c)                                  # without the sequences that have no rows
    rows = [b for b, n in enumerate(c.new) if n > 0]
    c.new, c.lens, c.table = [c.new[b] for b in rows], [c.lens[b] for b in rows], c.table[rows]
    want, tol = ref.attention(c, q, scale, softcap)
    tol = tol + UNIT[q.dtype] * (want.abs() + tol) + TINY[q.dtype]
    err = (got.cpu().double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}; first {bad.nonzero()[:3].tolist()}"


def _ragged(B, most_new, empty, seed, long=()):
    """(older, new) of B sequences, some without new tokens (some of those without any), a few long."""
    r = random.Random(seed)
    older = [r.randint(0, 90) for _ in range(B)]
    new = [0 if r.random() < empty else r.randint(1, most_new) for _ in range(B)]
    new[0] = most_new
    for b, n in long:
        older[b], new[b] = n, max(new[b], 1)
    older = [0 if new[b] == 0 and b % 2 else older[b] for b in range(B)]
    return older, new


@pytest.mark.parametrize("B,most_new", [(33, 1), (129, 1), (300, 1), (150, 3)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention_of_many_sequences(dt, B, most_new):
    """Runs of the split kernel that are cut and joined, far along the batch too."""
    older, new = _ragged(B, most_new, 0.2, B, long=[(1, 1500), (B // 2, 900), (B - 2, 2100), (B - 1, 40)])
    c = ref.Cache(older, new, 2, 64, 32, seed=B, fill=0x7F)
    q = _randn(B, c.T, 6, 64).to(DT[dt])
    out = ops.cache_attention(q.cuda(), *c.args())
    _check(out, c, q, 0.125)
    assert torch.equal(out, ops.cache_attention(q.cuda(), *c.args()))


@pytest.mark.parametrize("B,heads,group,most", [(40, 1, 8, 220), (130, 2, 4, 150)])
def test_prompts_of_many_sequences(B, heads, group, most):
    """More (sequence, row tile) pairs than the kernel that ranks them takes."""
    older, new = _ragged(B, 24, 0.15, B + 1, long=[(3, 300), (B - 1, 500)])
    new[0], new[B // 2], new[B - 1] = most, most - 9, 130
    assert -(-most * group // 256) * B > 256
    c = ref.Cache(older, new, heads, 64, 16, seed=B, fill=0xFF)
    q = _randn(B, c.T, heads * group, 64).half()
    out = ops.cache_attention(q.cuda(), *c.args())
    _check(out, c, q, 0.125)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [192, 256])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_prompts_of_wide_heads(dt, D, softcap):
    c = ref.Cache([50, 0, 301, 7], [130, 77, 1, 240], 2, D, 32, seed=D, fill=0x7F)
    q = _randn(D, c.T, 6, D).to(DT[dt])
    out = ops.cache_attention(q.cuda(), *c.args(), softcap=softcap)
    _check(out, c, q, D ** -0.5, softcap)


@pytest.mark.parametrize("D,heads,group", [(64, 8, 4), (128, 8, 2), (96, 4, 8)])
def test_a_prompt_chunk_beside_single_tokens(D, heads, group):
    c = ref.Cache([700, 3, 60, 1200, 0, 250, 90, 500], [1, 1, 170, 1, 1, 1, 5, 1], heads, D, 16, seed=D)
    q = _randn(D, c.T, heads * group, D).bfloat16()
    args = c.args()
    out = ops.cache_attention(q.cuda(), *args)
    _check(out, c, q, D ** -0.5)
    # a table with room for much more, and the most new tokens left to the call
    args[4] = torch.cat([args[4], torch.full((8, 500), -1, dtype=torch.int32, device="cuda")], 1)
    _check(ops.cache_attention(q.cuda(), *args[:7]), c, q, D ** -0.5)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,most_new,q_heads", [(40, 3, 4), (100, 2, 8), (300, 1, 4), (70, 60, 61)])
def test_append_over_many_sequences(layout, B, most_new, q_heads):
    older, new = _ragged(B, most_new, 0.25, B)
    c = ref.Cache(older, new, 1, 64, 32, seed=B)
    rows = _randn(B, c.T, 2 + q_heads, 64).bfloat16().cuda()
    k, v, q = rows[:, :1], rows[:, 1:2], rows[:, 2:]
    table = ops.rotary_table(max(c.lens), 64)
    kc, vc, ks, vs, *rest = c.args()
    q_out = ops.cache_append(k, v, kc, vc, ks, vs, *rest, table=table, layout=layout, q=q)
    pos = torch.cat([torch.arange(a, a + n) for a, n in zip(older, new)]).int().cuda()
    assert torch.equal(q_out, ops.rotary(q, table, pos, layout))
    # each sequence by itself gives the same pages
    kc1, vc1, ks1, vs1, pages, lens, starts, _ = c.args()
    at = 0
    for b, n in enumerate(new):
        if n > 0:
            ops.cache_append(k[at: at + n], v[at: at + n], kc1, vc1, ks1, vs1, pages[b: b + 1].contiguous(),
                             lens[b: b + 1], table=table, layout=layout)
        at += n
    for x, y in ((kc, kc1), (vc, vc1), (ks, ks1), (vs, vs1)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 170, 3]])
def test_steps_captured_into_a_graph(new):
    """Append and attention, the lengths advanced inside the graph: three replays against three calls."""
    heads, group, D = 8, 4, 64
    c = ref.Cache([900, 5, 130], [3 * n for n in new], heads, D, 32, seed=1)
    T = sum(new)
    starts = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    table = ops.rotary_table(2000, D)
    rows = _randn(2, T, heads * (group + 2), D).bfloat16().cuda()
    q, k, v = rows[:, :heads * group], rows[:, heads * group: heads * (group + 1)], rows[:, heads * (group + 1):]
    add = torch.tensor(new, dtype=torch.int32).cuda()

    def step(cache, lens):
        lens += add
        pool = (*cache, lens, starts, max(new))
        turned = ops.cache_append(k, v, *pool, table=table, q=q)
        return ops.cache_attention(turned, *pool)

    def fresh():
        return c.args()[:5], torch.tensor([900, 5, 130], dtype=torch.int32).cuda()

    cache, lens = fresh()
    want = []
    for i in range(3):
        rows.copy_(_randn(10 + i, *rows.shape))
        want.append(step(cache, lens).clone())
    side = torch.cuda.Stream()
    other, other_lens = fresh()
    with torch.cuda.stream(side):                     # once outside, as graphs want
        step(*fresh())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(other, other_lens)
    for i in range(3):
        rows.copy_(_randn(10 + i, *rows.shape))
        graph.replay()
        assert torch.equal(out, want[i])
    for x, y in zip(cache, other):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def _calls(seed):
    """One caller's own inputs: a cut decode batch, prompts and a rotation, each with its result."""
    cases = []
    for older, new, heads, group, D in (([2500, 900], [1, 1], 2, 4, 128), ([100] * 4, [70, 3, 90, 33], 8, 4, 64)):
        c = ref.Cache(older, new, heads, D, 16, seed=seed)
        q, args = _randn(seed, c.T, heads * group, D).half().cuda(), c.args()
        cases.append((lambda q=q, args=args, **kw: ops.cache_attention(q, *args, **kw)))
    x, table = _randn(seed + 1, 300, 8, 64).half().cuda(), ops.rotary_table(300, 64)
    pos = torch.arange(300, dtype=torch.int32).cuda()
    cases.append(lambda **kw: ops.rotary(x, table, pos, **kw))
    return [(f, f()) for f in cases]


def test_two_streams_at_once():
    calls = [_calls(s) for s in (1, 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[] for _ in streams]
    for _ in range(20):
        for s, mine, out in zip(streams, calls, got):
            out += [(f(stream=s), want) for f, want in mine]
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(y, want) for y, want in out)


def test_two_threads_at_once():
    calls = [_calls(s) for s in (3, 4)]
    torch.cuda.synchronize()
    wrong, failed = [], []

    def run(mine):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    for f, want in mine:
                        if not torch.equal(f(), want):
                            wrong.append(f)
        except BaseException as e:                     # raised again below
            failed.append(e)

    threads = [threading.Thread(target=run, args=(mine,)) for mine in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and not wrong
