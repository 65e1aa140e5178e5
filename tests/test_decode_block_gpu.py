"""The decoder-block example: prompts and single tokens against a 64-bit block that rounds where
the operators round, over the cache that the appends left."""
import pytest
import torch

import decoder_ref as ref
from gemm_conv_chains_gb300 import ops

pytestmark = pytest.mark.gpu
RTOL = 2e-2        # the framework's bar for bf16 chains, |gpu - ref| <= RTOL * max(1, |ref|)


def _close(got, want):
    got = got.cpu().double()
    assert ((got - want).abs() <= RTOL * want.abs().clamp_min(1)).all(), (got - want).abs().max()


def _round(t):
    return t.to(torch.bfloat16).double()


def _block(block, cache, x, new):
    """The block in 64 bits: the cached keys and values are the ones the call wrote."""
    from examples import decode_block as ex
    w = {k: getattr(block, k).cpu().double() for k in ("wq", "wkv", "wo", "w0", "w1")}
    x = x.cpu().double()
    c = ref.Cache([n - m for n, m in zip(cache.lens, new)], new, ex.KV_HEADS, ex.HEAD, ex.PAGE)
    c.k, c.v, c.ks, c.vs = (t.cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale))
    c.table = cache.table
    pos = torch.cat([torch.arange(n - m, n) for n, m in zip(cache.lens, new)])
    cs = block.table.cpu().double()[pos]
    q = ref.turn(_round(x @ w["wq"]).view(-1, ex.HEADS, ex.HEAD), cs, "half")
    a, _ = ref.attention(c, _round(q), ex.HEAD ** -0.5)
    x = _round(x + _round(_round(a).reshape(-1, ex.WIDTH) @ w["wo"]))
    h = x @ w["w0"]
    h = _round(h * ((h + 3).clamp(0, 6) / 6))
    return _round(x + _round(h @ w["w1"]))


def test_prompts_then_tokens():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from examples import decode_block as ex
    ops.get_cache_error()
    new = [70, 1, 33, 128]
    block, cache = ex.DecoderBlock(positions=200, seed=3), ex.Pages(4, 20, 5)
    x = torch.randn(sum(new), ex.WIDTH, generator=torch.Generator().manual_seed(4)).bfloat16()
    y = block(x.cuda(), cache, new)
    want = _block(block, cache, x, new)
    _close(y, want)
    # what was cached: the last call's keys and values within half an e4m3 step of the page's
    # largest, and the rounding of the projection
    kv = _round(x.double() @ block.wkv.cpu().double()).view(-1, 2 * ex.KV_HEADS, ex.HEAD)
    pos = torch.cat([torch.arange(n) for n in new])
    k = ref.turn(kv[:, :ex.KV_HEADS], block.table.cpu().double()[pos], "half")
    c = ref.Cache([0] * 4, new, ex.KV_HEADS, ex.HEAD, ex.PAGE)
    c.k, c.v, c.ks, c.vs = (t.cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale))
    c.table, at = cache.table, 0
    for b, n in enumerate(new):
        for got, full in zip(c.values(b, n), (k, kv[:, ex.KV_HEADS:])):
            full = full[at: at + n].transpose(0, 1)
            assert ((got - full).abs() <= full.abs() * (2.0 ** -4 + 2.0 ** -7) +
                    full.abs().max() * 2.0 ** -9).all()
        at += n
    for _ in range(3):
        x = y[-4:].contiguous() * 0.25
        y = block(x, cache, [1] * 4)
        want = _block(block, cache, x, [1] * 4)
        _close(y, want)
    assert ops.get_cache_error()[0] == 0
