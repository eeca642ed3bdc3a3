"""Calls whose result has no history say so where a gradient is asked for. On the CPU: refused before the device is touched."""
import pytest
import torch

from dspark_draft_sampling_gb300 import api
from tests.test_kv_devices import cache, ints, on, world  # noqa: F401


def arguments(index=0, grad=False, **out):
    x = on(index, 4, 4, 64)
    x.requires_grad_(grad)
    return (x, ints(index, 4), api.RotaryTable(ints(index, 16, dtype=torch.int64))), out


@pytest.mark.parametrize("backward", [False, True])
def test_rotary_refuses_to_drop_a_gradient(world, backward):  # noqa: F811
    args, _ = arguments(grad=True)
    with pytest.raises(ValueError, match="backward=True"):
        api.rotary(*args, backward=backward, out=on(0, 4, 4, 64))
    plain, _ = arguments()
    out = on(0, 4, 4, 64).requires_grad_()
    with pytest.raises(ValueError, match="backward=True"):
        api.rotary(*plain, backward=backward, out=out)
    assert not world.calls


def test_rotary_without_a_gradient_asked_for(world):  # noqa: F811
    args, _ = arguments(grad=True)
    with torch.no_grad():
        api.rotary(*args, out=on(0, 4, 4, 64))
    detached = on(0, 4, 4, 64)
    api.rotary(detached, *args[1:], out=detached)
    assert len(world.calls) == 2


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_inside_a_function_with_history(layout):
    # y is linear in x, so <w, y(x)> is <dL/dx, x>: the sums agree to the roundings of 4 * 3 * 32 terms below 20
    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, positions, table):
            ctx.save_for_backward(positions)
            ctx.table = table
            return api.rotary(x, positions, table)

        @staticmethod
        def backward(ctx, dy):
            return api.rotary(dy, ctx.saved_tensors[0], ctx.table, backward=True), None, None

    gen = torch.Generator().manual_seed(5)
    x, w = (torch.randn((4, 3, 32), generator=gen).cuda() for _ in range(2))
    x.requires_grad_()
    positions = torch.tensor([0, 3, 500, 70000], dtype=torch.int32).cuda()
    table = api.RotaryTable(api.rotary_frequencies(16), layout=layout, amplitude=1.25)
    y = Turn.apply(x, positions, table)
    y.backward(w)
    left, right = (w.double() * y.double()).sum(), (x.grad.double() * x.double()).sum()
    assert abs(float((left - right).detach())) <= 4 * 3 * 32 * 20 * 2.0**-20
