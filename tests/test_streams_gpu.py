"""Calls on a stream of their own: where their outputs' memory comes from."""
import pytest
import torch

from gemm_conv_chains_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ops.lib()


def _pool(t):
    """The stream whose memory holds t."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


def _r(*shape):
    return torch.randn(*shape, device="cuda").half()


def _vector(n):
    return torch.rand(n, device="cuda") + 0.5


CALLS = {
    "b2b_gemm": lambda: (_r(256, 64), _r(64, 64), None, _r(64, 64), None),
    "b2b_gemm3": lambda: (_r(256, 64), _r(64, 64), None, _r(64, 64), None, _r(64, 64), None),
    "b2b_conv_nhwc": lambda: (_r(1, 8, 8, 64), _r(64, 3, 3, 64), None, _r(64, 64), None),
    "b2b_conv_nhwc_strided": lambda: (_r(1, 8, 8, 64), _r(64, 3, 3, 64), None, _r(64, 64), None),
    "conv_relu_maxpool": lambda: (_r(1, 8, 8, 64), _r(64, 3, 3, 64), None),
    "gemm_bias_act": lambda: (_r(256, 64), _r(64, 64), None),
    "conv_bias_act_nhwc": lambda: (_r(1, 8, 8, 64), _r(64, 3, 3, 64), None),
    "maxpool2x2_nhwc": lambda: (_r(1, 8, 8, 64),),
    "fold_batchnorm": lambda: (_r(64, 64), None, _vector(64), _vector(64), _vector(64), _vector(64)),
    "rotary_table": lambda: (100, 64),
    "rotary": lambda: (_r(5, 2, 64), ops.rotary_table(9, 64),
                       torch.arange(5, dtype=torch.int32, device="cuda")),
}


@pytest.mark.parametrize("name", CALLS)
def test_outputs_come_from_the_memory_of_the_stream_that_writes_them(name):
    side = torch.cuda.Stream()
    args = CALLS[name]()
    torch.cuda.synchronize()

    def pools(stream):
        out = getattr(ops, name)(*args, stream=stream)
        torch.cuda.synchronize()
        return {_pool(t) for t in (out if isinstance(out, tuple) else (out,))}

    for stream, pool in ((side, side.cuda_stream), (side.cuda_stream, side.cuda_stream), (None, 0), (0, 0),
                         (torch.cuda.default_stream(), 0)):
        assert pools(stream) == {pool}
    with torch.cuda.stream(side):
        assert pools(None) == {side.cuda_stream}
        assert pools(0) == {0}


def test_memory_that_runs_out_is_torch_s_error():
    """Rows that overlap: operands of some MB, outputs of 2 TB."""
    rows, head = 2 ** 20, 2 ** 20
    x = torch.zeros(rows * 8 + head, dtype=torch.float16, device="cuda").as_strided((rows, 1, head), (8, head, 1))
    positions = torch.zeros(rows, dtype=torch.int32, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        ops.rotary(x, ops.rotary_table(4, 64), positions)
    cache = [torch.zeros(1, 1, 16, 64, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)] + \
        [torch.ones(1, 1, device="cuda") for _ in range(2)] + \
        [torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")]
    q = x[:, :, :64].expand(rows, head, 64).as_strided((rows, head // 64, 64), (8, 64, 1))
    assert q.numel() == rows * head
    with pytest.raises(torch.OutOfMemoryError):
        ops.cache_attention(q, *cache)
    torch.cuda.synchronize()
