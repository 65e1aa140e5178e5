"""Outputs that overlap what the call still reads are refused before anything is launched; rows side by
side in one buffer, and the in-place forms, are not."""
import pytest
import torch

from gemm_conv_chains_gb300 import ops

import decoder_ref as ref

pytestmark = pytest.mark.gpu
UNSUPPORTED = 4


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ops.lib()
    ops.get_cache_error()
    yield
    assert ops.get_cache_error()[0] == 0


def _rows(T, heads, D=64, seed=0):
    return torch.randn(T, heads, D, generator=torch.Generator().manual_seed(seed)).half().cuda()


def _refused(call):
    with pytest.raises(ops.B2BError) as e:
        call()
    assert e.value.status == UNSUPPORTED


def test_attention_into_its_queries():
    c = ref.Cache([900, 30, 5], [1, 1, 1], 2, 64, 16)
    args = c.args()
    buf = torch.zeros(3 * 4 * 64 * 4, dtype=torch.float16, device="cuda")
    q = buf[:768].view(3, 4, 64)
    q.copy_(_rows(3, 4))
    want = ops.cache_attention(q, *args)
    _refused(lambda: ops.cache_attention(q, *args, out=q))
    _refused(lambda: ops.cache_attention(q, *args, out=buf[64:832].view(3, 4, 64)))
    assert torch.equal(ops.cache_attention(q, *args, out=buf[768:1536].view(3, 4, 64)), want)
    wide = torch.zeros(3, 32, 64, dtype=torch.float16, device="cuda")          # a fused projection's rows
    wide[:, :4] = q
    gap = wide.view(-1)[4 * 64: 4 * 64 + 768].view(3, 4, 64)                   # between the first two rows' q
    assert torch.equal(ops.cache_attention(wide[:, :4], *args, out=gap), want)
    _refused(lambda: ops.cache_attention(wide[:, :4], *args, out=wide.view(-1)[1536:2304].view(3, 4, 64)))


def test_rotary_into_rows_that_overlap():
    table, pos = ops.rotary_table(16, 64), torch.arange(5, dtype=torch.int32, device="cuda")
    rows = _rows(5, 12)
    keep = rows.clone()
    want = ops.rotary(rows[:, :4], table, pos)
    _refused(lambda: ops.rotary(rows[:, :4], table, pos, out=rows[:, 2:6]))
    _refused(lambda: ops.rotary(rows[:4, :4], table, pos[:4], out=rows[1:, :4]))
    _refused(lambda: ops.rotary(rows[:, :4], table, pos, out=rows.view(-1)[:1280].view(5, 4, 64)))
    assert torch.equal(rows, keep)
    ops.rotary(rows[:, :4], table, pos, out=rows[:, 6:10])                     # beside it
    assert torch.equal(rows[:, 6:10], want) and torch.equal(rows[:, :6], keep[:, :6])
    ops.rotary(rows[:, :4], table, pos, out=rows[:, :4])                       # in place
    assert torch.equal(rows[:, :4], want)


def test_append_s_queries_into_rows_that_overlap():
    c = ref.Cache([0, 9], [2, 2], 2, 64, 16)
    args = c.args()
    table = ops.rotary_table(16, 64)
    rows = _rows(4, 12)                                                        # q, k, v: 4, 2, 2 heads; 4 more
    q, k, v = rows[:, :4], rows[:, 4:6], rows[:, 6:8]
    keep, codes = rows.clone(), args[0].clone()
    for out in (rows[:, 1:5], rows[:, 4:8], rows[:, 5:9], rows[:, 7:11]):
        _refused(lambda: ops.cache_append(k, v, *args, table=table, q=q, q_out=out))
    assert torch.equal(rows, keep) and torch.equal(codes.view(torch.uint8), args[0].view(torch.uint8))
    want = ops.cache_append(k, v, *args, table=table, q=q)
    assert torch.equal(ops.cache_append(k, v, *args, table=table, q=q, q_out=rows[:, 8:12]), want)
    assert torch.equal(ops.cache_append(k, v, *args, table=table, q=q, q_out=q), want)
