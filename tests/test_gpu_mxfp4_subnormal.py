"""MXFP4 blocks whose largest magnitude is below the fp32 normal range: the scale
code is 0, the step 2^-127, and the codes are v / step to nearest even, as for
every other block; only a block of zeros has zero codes alone.

Every value here is a multiple of 2^-133 below 2^-126 (bf16's and fp32's
subnormals), so v / step is exact and the expected codes need no tolerance."""
import pytest
import torch

from mixture_experts_layer_schedule_gb300 import FP4Linear, FP4Tensor

from gpu_helpers import dev
from test_gpu_ffn import E32, rounding

pytestmark = pytest.mark.gpu

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0], dtype=torch.float64)  # v < 2^-126: at most 2 steps
STEP = 2.0 ** -127


def expected(units):
    """Values of codes of units * 2^-133 (exact integers), ties to the even code."""
    q = units.abs().double() / 64.0  # in steps of 2^-127
    d = (q.unsqueeze(-1) - GRID).abs()
    lo = d.argmin(-1)
    tie = (lo + 1 < len(GRID)) & (d.gather(-1, lo.unsqueeze(-1)).squeeze(-1)
                                  == d.gather(-1, (lo + 1).clamp(max=len(GRID) - 1).unsqueeze(-1)).squeeze(-1))
    idx = torch.where(tie & (lo % 2 == 1), lo + 1, lo)
    return idx, torch.sign(units.double()) * GRID[idx] * STEP


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_blocks_below_the_normal_range(dtype):
    rows, cols = 5, 256
    gen = torch.Generator().manual_seed(3)
    units = torch.randint(-127, 128, (rows, cols), generator=gen)  # bf16: 7 bits below 2^-126
    units[0] = torch.arange(cols) - 128  # every value, every tie
    units[0, 0] = 0
    units[1, :32] = 0                    # a block of zeros between others
    units[2] = torch.where(units[2].abs() < 16, 0, units[2] % 16)  # rounds to zeros alone
    x = (units.double() * 2.0 ** -133).to(torch.float32)
    assert torch.equal(x.double(), units.double() * 2.0 ** -133)
    x = x.to(dtype)
    assert torch.equal(x.double(), units.double() * 2.0 ** -133)
    t = FP4Tensor(rows, cols, format="mxfp4").quantize(x.to(dev()))
    idx, val = expected(units)
    packed = t.q.cpu()
    nib = torch.stack((packed & 15, packed >> 4), -1).reshape(rows, cols)
    assert torch.equal((nib & 7).long(), idx)
    assert torch.equal((nib >> 3).bool(), units < 0)
    assert not t.s.any()  # scale code 0, padding included
    assert torch.equal(t.dequantize(dtype=torch.float32).cpu().double(), val)


def test_the_step_to_the_normal_range():
    """Blocks on either side of 2^-126 and of 2^-125, where the step doubles."""
    for top in (2.0 ** -127, 1.5 * 2.0 ** -127, 2.0 ** -126, 1.75 * 2.0 ** -126, 2.0 ** -125, 2.0 ** -124, 2.0 ** -123):
        x = torch.zeros((1, 32), dtype=torch.float32)
        x[0, 3], x[0, 7] = top, -top / 2
        code = max(int(torch.frexp(torch.tensor(top, dtype=torch.float64)).exponent) - 1 - 2 + 127, 0)
        t = FP4Tensor(1, 32, format="mxfp4").quantize(x.to(dev()))
        assert int(t.s[0]) == code
        # top is 1 to 1.75 times a power of two that is 0.5, 1, 2 or 4 steps: exact but for
        # 1.5 and 1.75 of steps that E2M1 lacks
        q = torch.tensor([top, top / 2], dtype=torch.float64) / 2.0 ** (code - 127)
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
        want = []
        for v in q:
            d = (grid - v).abs()
            best = [i for i in range(8) if d[i] == d.min()]
            want.append(grid[min(best, key=lambda i: i % 2)] * 2.0 ** (code - 127))
        got = t.dequantize(dtype=torch.float32).cpu().double()
        assert got[0, 3] == want[0] and got[0, 7] == -want[1], top


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("M", [3, 40])
def test_products_of_such_activations(M, kernel):
    """Large weights bring them back into range: the bound of test_gpu_fp4.py."""
    N, K = 72, 288
    gen = torch.Generator().manual_seed(M)
    x = (torch.randint(-127, 128, (M, K), generator=gen).double() * 2.0 ** -133).to(torch.bfloat16).to(dev())
    w = (torch.randint(-6, 7, (N, K), generator=gen).double() * 2.0 ** 118).to(torch.bfloat16).to(dev())
    wq = FP4Tensor(N, K, format="mxfp4").quantize(w)
    xd = FP4Tensor(M, K, format="mxfp4").quantize(x).dequantize(dtype=torch.float32).double()
    wd = wq.dequantize(dtype=torch.float32).double()
    assert xd.any()
    ref = xd @ wd.t()
    y = FP4Linear(M, N, K, format="mxfp4", kernel=kernel).forward(x, wq)
    bound = rounding(ref, torch.bfloat16) + E32 * (xd.abs() @ wd.abs().t())
    assert ((y.double() - ref).abs() <= bound).all()
