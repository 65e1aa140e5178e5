"""Rotary positions under autograd: the gradient is the inverse rotation, whatever the gradient that
arrives looks like."""
import pytest
import torch

from gemm_conv_chains_gb300 import ops

import decoder_ref as ref
from decoder_ref import TINY, UNIT

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ops.lib()
    ops.get_cache_error()
    yield
    assert ops.get_cache_error()[0] == 0


def _case(T, H, D, rot, gain=1.0, pad=0):
    g = torch.Generator().manual_seed(T)
    rows = torch.randn(T, H + pad, D, generator=g).half().cuda()
    table = ops.rotary_table(500, rot, gain=gain)
    positions = torch.randint(500, (T,), generator=g, dtype=torch.int32).cuda()
    return rows, table, positions


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("gain", [1.0, 1.25])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 64, 64), (7, 3, 96, 48), (9001, 12, 64, 32)])
def test_the_gradient_is_the_inverse_rotation(layout, inverse, gain, T, H, D, rot):
    rows, table, positions = _case(T, H, D, rot, gain)
    w = torch.randn_like(rows)
    x = rows.clone().requires_grad_(True)
    y = ops.rotary(x, table, positions, layout, inverse)
    assert y.requires_grad
    assert torch.equal(y.detach(), ops.rotary(rows, table, positions, layout, inverse))
    y.backward(w)
    assert torch.equal(x.grad, ops.rotary(w, table, positions, layout, not inverse))
    # and by the formula, differentiated in 64 bits
    xx = rows.cpu().double().requires_grad_(True)
    cs = table.cpu().double()[positions.cpu().long()]
    ref.turn(xx, cs, layout, inverse).backward(w.cpu().double())
    tol = UNIT[torch.float16] * xx.grad.abs() + 2.0 ** -22 * 16 + TINY[torch.float16]
    assert ((x.grad.cpu().double() - xx.grad).abs() <= tol).all()


def test_gradients_that_are_broadcast_or_in_another_order():
    rows, table, positions = _case(19, 4, 64, 64)
    for back in (lambda y: y.sum(), lambda y: y[..., 0].sum(), lambda y: (y.transpose(0, 1) * w).sum()):
        w = torch.randn(4, 19, 64, device="cuda").half()
        x = rows.clone().requires_grad_(True)
        back(ops.rotary(x, table, positions)).backward()
        y = rows.clone().requires_grad_(True)
        back(y).backward()
        assert torch.equal(x.grad, ops.rotary(y.grad.contiguous(), table, positions, inverse=True))


def test_through_the_slices_of_a_fused_projection():
    rows, table, positions = _case(33, 4, 64, 32, pad=2)
    fused = rows.clone().requires_grad_(True)
    y = ops.rotary(fused[:, :4], table, positions)
    w = torch.randn_like(y)
    (y * w).sum().backward()
    assert torch.equal(fused.grad[:, :4], ops.rotary(w, table, positions, inverse=True))
    assert not fused.grad[:, 4:].any()


def test_the_gradient_can_be_differentiated():
    rows, table, positions = _case(5, 2, 64, 64)
    x, w, v = rows.clone().requires_grad_(True), torch.randn_like(rows).requires_grad_(True), \
        torch.randn_like(rows)
    grad, = torch.autograd.grad(ops.rotary(x, table, positions), x, w, create_graph=True)
    back, = torch.autograd.grad(grad, w, v)
    assert torch.equal(back, ops.rotary(v, table, positions))


def test_without_a_gradient_nothing_is_recorded():
    rows, table, positions = _case(5, 2, 64, 64)
    assert not ops.rotary(rows, table, positions).requires_grad
    x = rows.clone().requires_grad_(True)
    with torch.no_grad():
        assert not ops.rotary(x, table, positions).requires_grad
        assert not ops.rotary(x, table, positions, out=torch.empty_like(rows)).requires_grad


def test_refusals():
    rows, table, positions = _case(5, 2, 64, 64)
    x = rows.clone().requires_grad_(True)
    with pytest.raises(ValueError, match="out is given"):
        ops.rotary(x, table, positions, out=torch.empty_like(rows))
    with pytest.raises(ValueError, match="out is given"):
        ops.rotary(rows, table, positions, out=x)
    with pytest.raises(ValueError, match="table requires"):
        ops.rotary(rows, table.clone().requires_grad_(True), positions)
    with pytest.raises(ValueError, match="positions has shape"):
        ops.rotary(x, table, positions[:3])
