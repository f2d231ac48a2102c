"""The 4-bit block's tensor scales of its input and of its inner activations."""
import pytest
import torch

from mixture_experts_layer_schedule_gb300 import FP4GatedFFN, FP4Linear, FP4Tensor, GatedFFN, MoEError

from gpu_helpers import dev

pytestmark = pytest.mark.gpu


def block(N, H, I, x_size):
    gen = torch.Generator(device=dev()).manual_seed(N)
    x = (torch.randn((N, H), generator=gen, device=dev()) * x_size).to(torch.bfloat16)
    w = [(torch.randn(s, generator=gen, device=dev()) * s[1] ** -0.5).to(torch.bfloat16)
         for s in ((I, H), (I, H), (H, I))]
    return x, w


@pytest.mark.parametrize("N", [1, 30, 300])
def test_small_activations_keep_their_bits(N):
    """Inputs of 2^-12 give inner activations near 2^-26: with tensor scales of 1
    all of them are zero, with fitting ones the block is as close to the 16-bit block as
    for inputs of ordinary size. The bound is that of test_gpu_shared_expert.py: three
    products of operands with the 4-bit error e each, sqrt(6) e, twice that."""
    H, I = 512, 256
    x, w = block(N, H, I, 2.0 ** -12)
    q = FP4GatedFFN.quantize_weights(*w)
    want = GatedFFN(N, H, I, training=False).forward_inference(x, *w).float()
    assert not FP4GatedFFN(N, H, I).forward(x, *q).any()
    a, b = 2.0 ** -21, 2.0 ** -34  # about max / 2688 of x and of A
    f = FP4GatedFFN(N, H, I, x_scale=a, act_scale=b)
    got = f.forward(x, *q)
    n = torch.randn((64, 512), device=dev())
    e = float((FP4Tensor.of_weight(n).dequantize(dtype=torch.float32) - n).norm() / n.norm())
    assert e < 0.15 and float((got.float() - want).norm() / want.norm()) < 2 * (6 * e * e) ** 0.5
    up, down = FP4Linear(N, I, H, x_scale=a), FP4Linear(N, H, I, x_scale=b)
    assert torch.equal(got, down.forward(up.forward_gated(x, q[0], q[1]), q[2]))
    assert f.device_error() == 0


def test_mxfp4_has_no_tensor_scale():
    x, w = block(4, 64, 64, 1.0)
    q = FP4GatedFFN.quantize_weights(*w, format="mxfp4")
    FP4GatedFFN(4, 64, 64, format="mxfp4").forward(x, *q)
    for kw in (dict(x_scale=2.0), dict(act_scale=0.5)):
        with pytest.raises(MoEError):
            FP4GatedFFN(4, 64, 64, format="mxfp4", **kw).forward(x, *q)


def test_error_words_can_be_cleared():
    """Both products' error words, set here on the host's behalf, read as zero again."""
    f = FP4GatedFFN(4, 64, 64)
    for product in (f.gate_up, f.down):
        product.ws[:4].view(torch.int32).fill_(3)
        assert f.device_error() == 3
        f.clear_device_error()
        assert f.device_error() == 0 and product.device_error() == 0
