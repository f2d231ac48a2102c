"""4-bit matrices made and read back on a stream of the caller's: everything that
such a call does, its memory included, belongs to that stream."""
import pytest
import torch

from mixture_experts_layer_schedule_gb300 import FP4Tensor

from gpu_helpers import dev

pytestmark = pytest.mark.gpu

BUSY = 50_000_000  # clock cycles: about 25 ms, the current stream is through long before


def late_weight(stream, small, large):
    """A weight that holds `small` until `stream`, busy for a while, writes `large`."""
    w = torch.full((128, 128), small, device=dev(), dtype=torch.bfloat16)
    new = torch.full((128, 128), large, device=dev(), dtype=torch.bfloat16)
    FP4Tensor.of_weight(new)  # no lazy loading behind the sleep
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(BUSY)
        w.copy_(new)
    return w, new


@pytest.mark.parametrize("raw", [False, True])
def test_weight_written_on_the_stream_that_quantises_it(raw):
    s = torch.cuda.Stream()
    w, new = late_weight(s, 2.0 ** -12, 24.0)
    t = FP4Tensor.of_weight(w, stream=s.cuda_stream if raw else s)
    s.synchronize()
    want = FP4Tensor.of_weight(new)
    torch.cuda.synchronize()
    assert t.scale == want.scale and torch.equal(t.q, want.q) and torch.equal(t.s, want.s)
    assert torch.equal(t.dequantize(dtype=torch.float32), new.float())


def test_read_back_takes_memory_of_its_own_stream():
    """A block that the current stream still uses is not handed to a read-back on
    another stream, which would write it first."""
    rows = cols = 1024
    ones = torch.ones((rows, cols), device=dev(), dtype=torch.bfloat16)
    t = FP4Tensor(rows, cols, format="mxfp4").quantize(ones)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    t.dequantize(torch.empty_like(ones), stream=s)  # no lazy loading below
    torch.cuda.synchronize()
    torch.cuda.empty_cache()  # the next block of this size is the one freed below
    late = torch.empty((rows, cols), device=dev(), dtype=torch.bfloat16)
    torch.cuda._sleep(BUSY)
    late.fill_(7.0)  # runs after the sleep
    del late         # its block may be reused by work of the current stream only
    out = t.dequantize(stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, ones)


def test_default_stream_by_its_handle():
    w = torch.randn((32, 64), device=dev()).to(torch.bfloat16)
    t = FP4Tensor.of_weight(w, "mxfp4", stream=0)
    torch.cuda.synchronize()
    assert torch.equal(t.dequantize(stream=0), FP4Tensor.of_weight(w, "mxfp4").dequantize())
