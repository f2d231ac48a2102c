"""Calls whose operand is the object's own result, which the call writes: they come up
when one object serves several layers and the result of one call is handed to the
next. The results are those of calls with a copy, up to the order of fp32 sums where
another kernel is chosen (the bounds of test_gpu_fp4.py)."""
import pytest
import torch

from mixture_experts_layer_schedule_gb300 import FP4Linear, GatedFFN

import test_gpu_fp4 as fp4
from gpu_helpers import dev
from test_gpu_ffn import E32, act64, rounding

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M", [1, 5, 32, 77, 700])
def test_4_bit_products_of_their_own_result(M, fmt):
    """Wide enough that many CTAs read x while others are through."""
    K = N = 4096
    x, xq, (w0, w1), (d0, d1) = fp4.operands(M, N, K, fmt, BF, M, 2)
    lin = FP4Linear(M, N, K, format=fmt)
    g, eg = xq @ d0.t(), E32 * (xq.abs() @ d0.abs().t())
    u, eu = xq @ d1.t(), E32 * (xq.abs() @ d1.abs().t())
    h, _ = act64(g, "silu")
    for _ in range(5):
        lin.y.copy_(x)
        fp4.check(lin.forward(lin.y, w0), g, rounding(g, BF) + eg)
        lin.y.copy_(x)
        fp4.check(lin.forward_gated(lin.y, w0, w1), h * u,
                  rounding(h * u, BF) + 1.2 * (u.abs() * eg + h.abs() * eu) + E32 * (h * u).abs())
    assert lin.device_error() == 0


def test_4_bit_product_of_a_part_of_its_result():
    M, N, K = 3, 512, 256
    x, xq, (w,), (d,) = fp4.operands(M, N, K, "nvfp4", BF, 2, 1)
    lin = FP4Linear(M, N, K)
    lin.y[:, K:].copy_(x)
    y = lin.forward(lin.y[:, K:], w)
    fp4.check(y, xq @ d.t(), rounding(xq @ d.t(), BF) + E32 * (xq.abs() @ d.abs().t()))


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
