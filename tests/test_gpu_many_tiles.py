"""Sizes at which every SM pair walks several tiles and the quantiser several
column steps: the second accumulator, wrapped rings, staging buffers under
outstanding stores, and loads for the next tile under the present one's
epilogue. The bounds are those of test_gpu_ffn.py and test_gpu_fp4.py; sums over
N tokens run to 8003 terms, so the weight gradients' bound, whose fp32 term is
stated for 4096, is doubled."""
import pytest
import torch

from mixture_experts_layer_schedule_gb300 import FP4Linear, FP4Tensor, GatedFFN

import test_gpu_fp4 as fp4
from gpu_helpers import dev
from test_gpu_ffn import E32, act64, backward_ref, check, draw, forward_ref, rounding

pytestmark = pytest.mark.gpu


# 8003 x 1288 x 1032 in tiles of 256 x 256: gate/up 32 x 9, down and dX 32 x 6, the
# activation gradient 32 x 5 tiles, the weight gradients 90 over 76 pairs; ragged on
# every side.
@pytest.mark.parametrize("dtype,kind,grad_dtype", [(torch.bfloat16, "silu", torch.float32),
                                                   (torch.float16, "gelu", torch.float16)])
def test_dense_block(dtype, kind, grad_dtype):
    N, H, I = 8003, 1288, 1032
    d = draw(N, H, I, dtype, seed=5, pad=8)
    d["dy"] *= 0.125
    f = GatedFFN(N, H, I, dtype=dtype, activation=kind, grad_dtype=grad_dtype, kernel=1)
    args = (d["x"], d["wg"], d["wu"], d["wd"])
    y = f.forward(*args)
    grads = f.backward(d["dy"], *args)
    assert f.device_error() == 0
    ref = forward_ref(d, kind, dtype)
    for name, got in (("g", f.g), ("u", f.u), ("a", f.a), ("y", y)):
        check(name, got, ref[name])
    back = backward_ref(d, (f.g, f.u, f.a), kind, dtype, grad_dtype)
    check("dx", grads.dx, back["dx"])
    for name in ("dw_gate", "dw_up", "dw_down"):
        check(name, getattr(grads, name), (back[name][0], 2.0 * back[name][1]))
    first = {k: getattr(grads, k).clone() for k in back}
    y0 = y.clone()
    f.y.fill_(float("nan"))
    assert torch.equal(f.forward_inference(*args), y0)
    f.backward(d["dy"], *args)
    torch.cuda.synchronize()
    assert all(torch.equal(getattr(grads, k), v) for k, v in first.items()) and f.device_error() == 0


# 20 x 9 tiles linear, 20 x 17 gated; four and nine k-blocks against a ring of five.
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("K", [800, 2208])
def test_4_bit_products(K, fmt):
    M, N = 5003, 2056
    dtype, kind = (torch.float16, "gelu") if K == 800 else (torch.bfloat16, "silu")
    x, xq, (w0, w1), (d0, d1) = fp4.operands(M, N, K, fmt, dtype, K, 2, pad=8)
    lin = FP4Linear(M, N, K, format=fmt, dtype=dtype, activation=kind, kernel=1)
    g, eg = xq @ d0.t(), E32 * (xq.abs() @ d0.abs().t())
    u, eu = xq @ d1.t(), E32 * (xq.abs() @ d1.abs().t())
    y = lin.forward(x, w0).clone()
    fp4.check(y, g, rounding(g, dtype) + eg)
    h, _ = act64(g, kind)
    ref = h * u
    a = lin.forward_gated(x, w0, w1).clone()
    fp4.check(a, ref, rounding(ref, dtype) + 1.2 * (u.abs() * eg + h.abs() * eu) + E32 * ref.abs())
    assert torch.equal(lin.forward(x, w0), y) and torch.equal(lin.forward_gated(x, w0, w1), a)
    assert lin.device_error() == 0


# 516 row groups leave three CTAs a row group (two steps of 768 columns, the second
# ragged); 128 leave ten (two steps of 2560).
@pytest.mark.parametrize("rows,cols,dtype,fmt,ts", [(16385, 1056, torch.bfloat16, "nvfp4", 0.375),
                                                    (16385, 1056, torch.float32, "mxfp4", 1.0),
                                                    (4001, 4128, torch.float16, "nvfp4", 1.0)])
def test_quantiser_walks_its_columns(rows, cols, dtype, fmt, ts):
    x = fp4.values(rows, cols, dtype, seed=rows)
    t = FP4Tensor(rows, cols, format=fmt, scale=ts)
    t.s.fill_(0xAB)
    t.quantize(x)
    idx, sign, code, val = fp4.reference(x, fmt, ts)
    packed = t.q.cpu()
    nib = torch.stack((packed & 15, packed >> 4), -1).reshape(rows, cols)
    assert torch.equal(nib & 7, idx.to(torch.uint8)) and torch.equal((nib >> 3).bool(), sign)
    got = fp4.scale_bytes(t)
    assert torch.equal(got[:rows, : code.shape[1]].int(), code.int())
    assert not got[rows:].any() and not got[:, code.shape[1]:].any()
    assert torch.equal(t.dequantize(dtype=torch.float32).cpu(), val.float())


# ---- a tensor scale of the activations -----------------------------------------


@pytest.mark.parametrize("kernel", [0, 1, 2])
@pytest.mark.parametrize("M,N,K", [(1, 136, 512), (17, 264, 1056), (77, 264, 544), (300, 520, 768)])
@pytest.mark.parametrize("x_scale", [0.375, 2.0 ** -9])
def test_tensor_scale_of_the_activations(M, N, K, x_scale, kernel):
    """Activations small enough that a tensor scale of 1 would lose them. The
    product with the tensor scales is one more fp32 rounding of each, and the
    decoded operands are rounded by another: covered by the fp32 term."""
    gen = torch.Generator(device=dev()).manual_seed(M)
    x = (torch.randn((M, K), generator=gen, device=dev()) * 3.0 * x_scale).to(torch.bfloat16)
    ws = [FP4Tensor(N, K, scale=0.0007).quantize((torch.randn((N, K), generator=gen, device=dev()) * K ** -0.5)
                                                 .to(torch.bfloat16)) for _ in range(2)]
    xq = FP4Tensor(M, K, scale=x_scale).quantize(x).dequantize(dtype=torch.float32).double()
    d0, d1 = (w.dequantize(dtype=torch.float32).double() for w in ws)
    g, eg = xq @ d0.t(), E32 * (xq.abs() @ d0.abs().t())
    u, eu = xq @ d1.t(), E32 * (xq.abs() @ d1.abs().t())
    lin = FP4Linear(M, N, K, x_scale=x_scale, kernel=kernel)
    fp4.check(lin.forward(x, ws[0]), g, rounding(g, torch.bfloat16) + eg)
    h, _ = act64(g, "silu")
    ref = h * u
    fp4.check(lin.forward_gated(x, *ws), ref,
              rounding(ref, torch.bfloat16) + 1.2 * (u.abs() * eg + h.abs() * eu) + E32 * ref.abs())
    assert lin.device_error() == 0
