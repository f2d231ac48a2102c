"""What an FP4Tensor hands to the library follows its public q, s and scale (no GPU)."""
import pytest
import torch

from mixture_experts_layer_schedule_gb300 import FP4Tensor, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def handed(t):
    return t.operand.q, t.operand.s, t.operand.scale


def test_operand_follows_what_is_set():
    t = FP4Tensor(40, 96, scale=0.5, device="cpu")
    assert handed(t) == (t.q.data_ptr(), t.s.data_ptr(), 0.5) and t.scale == 0.5
    t.scale = 0.25
    assert handed(t)[2] == 0.25 and t.scale == 0.25
    q, s = torch.zeros_like(t.q), torch.ones_like(t.s)
    t.q, t.s = q, s
    assert t.q is q and t.s is s and handed(t) == (q.data_ptr(), s.data_ptr(), 0.25)
    assert t._operand._obj is t.operand  # the products take the same struct


def test_buffers_of_other_sizes_are_refused():
    t = FP4Tensor(40, 96, device="cpu")
    before = handed(t)
    for bad in (torch.zeros((40, 96), dtype=torch.uint8), torch.zeros((40, 48), dtype=torch.int8),
                torch.zeros((48, 40), dtype=torch.uint8).t(), torch.empty((40, 48), dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="q: expected"):
            t.q = bad
    for bad in (t.s[:-1], t.s.view(torch.int8), t.s.reshape(2, -1)):
        with pytest.raises(ValueError, match="s: expected"):
            t.s = bad
    assert handed(t) == before


@pytest.mark.gpu
def test_products_use_what_is_set():
    from mixture_experts_layer_schedule_gb300 import FP4Linear
    x = torch.randn((3, 64), device="cuda").to(torch.bfloat16)
    w = torch.randn((16, 64), device="cuda").to(torch.bfloat16)
    a, b = FP4Tensor.of_weight(w), FP4Tensor.of_weight(-2 * w)
    lin = FP4Linear(3, 16, 64)
    y = lin.forward(x, a).clone()
    stored = FP4Tensor(16, 64)
    stored.q, stored.s, stored.scale = a.q.clone(), a.s.clone(), a.scale
    assert torch.equal(lin.forward(x, stored), y)
    stored.scale = 4.0 * a.scale  # a power of two: exact
    assert torch.equal(lin.forward(x, stored), 4.0 * y)
    assert torch.equal(stored.dequantize(dtype=torch.float32), 4.0 * a.dequantize(dtype=torch.float32))
    stored.q, stored.s, stored.scale = b.q, b.s, b.scale
    assert torch.equal(lin.forward(x, stored), lin.forward(x, b))
