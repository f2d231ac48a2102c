"""Calls whose operand is the object's own result, which the call writes: they come up
when one object serves several layers and the result of one call is handed to the
next. The results are those of calls with a copy."""
import pytest
import torch

from mixture_experts_layer_schedule_gb300 import GatedFFN

from gpu_helpers import dev

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("N", [40, 1003])
def test_two_layers_through_one_dense_block(N, kernel):
    H, I = 256, 128
    gen = torch.Generator(device=dev()).manual_seed(N)
    x, dy = (torch.randn((N, H), generator=gen, device=dev()).to(BF) for _ in range(2))
    w = [(torch.randn(s, generator=gen, device=dev()) * s[1] ** -0.5).to(BF) for s in ((I, H), (I, H), (H, I))]
    one, a, b = (GatedFFN(N, H, I, kernel=kernel) for _ in range(3))
    y1 = a.forward(x, *w)
    y2 = b.forward(y1, *w)
    assert torch.equal(one.forward(one.forward(x, *w), *w), y2)
    names = ("dx", "dw_gate", "dw_up", "dw_down")
    db = b.backward(dy, y1, *w)
    da = a.backward(db.dx, x, *w)
    one.backward(dy, y1, *w, saved=(b.g, b.u, b.a))
    g = one.backward(one.grads.dx, x, *w, saved=(a.g, a.u, a.a))
    for name in names:
        assert torch.equal(getattr(g, name), getattr(da, name)), name
    # x in the place of dx
    one.grads.dx.copy_(x)
    g = one.backward(db.dx, one.grads.dx, *w, saved=(a.g, a.u, a.a))
    for name in names:
        assert torch.equal(getattr(g, name), getattr(da, name)), name
    assert one.device_error() == 0
