"""A launch that fails is reported by the call that made it, and by no later one: CUDA
keeps the error of a failed launch for whoever asks next, and the routed layer's
launches ask.

The failure is one of the host's, before anything reaches the GPU: a stream whose
capture was ended by an operation that captures do not allow refuses launches."""
import contextlib
import ctypes

import pytest
import torch

from mixture_experts_layer_schedule_gb300 import FP4Linear, FP4Tensor, GatedFFN, MoEError, MoELayer, _lib

from gpu_helpers import dev

pytestmark = pytest.mark.gpu

RELAXED = 2  # cudaStreamCaptureModeRelaxed: other streams and threads go on as usual


@contextlib.contextmanager
def broken_stream():
    lib = _lib.load()  # the CUDA runtime that the library is linked to
    s = torch.cuda.Stream()
    h = ctypes.c_void_p(s.cuda_stream)
    assert lib.cudaStreamBeginCapture(h, RELAXED) == 0
    assert lib.cudaStreamSynchronize(h) != 0  # not allowed: the capture is invalid now
    lib.cudaGetLastError()
    try:
        yield s
    finally:
        graph = ctypes.c_void_p()
        assert lib.cudaStreamEndCapture(h, ctypes.byref(graph)) != 0 and not graph.value
        lib.cudaGetLastError()


def test_no_error_is_left_for_the_next_call():
    lib = _lib.load()
    bf = dict(device=dev(), dtype=torch.bfloat16)
    x, wg, wd = torch.ones((4, 256), **bf), torch.ones((128, 256), **bf), torch.ones((256, 128), **bf)
    t, f, lin = FP4Tensor(128, 256), GatedFFN(4, 256, 128), FP4Linear(4, 128, 256)
    layer = MoELayer(64, 256, 256, 8, 2, device=dev())
    logits, bias = torch.randn((64, 8), device=dev()), torch.zeros(8, device=dev())
    out = torch.empty((128, 256), **bf)
    calls = dict(quantize=lambda s: t.quantize(wg, stream=s),
                 dequantize=lambda s: t.dequantize(out, stream=s),
                 linear=lambda s: lin.forward(x, t, stream=s),
                 forward=lambda s: f.forward(x, wg, wg, wd, stream=s),
                 backward=lambda s: f.backward(x, x, wg, wg, wd, stream=s),
                 clear=lambda s: f.clear_device_error(stream=s),
                 clear4=lambda s: lin.clear_device_error(stream=s))
    torch.cuda.synchronize()
    with broken_stream() as s:
        for name, call in calls.items():
            with pytest.raises(MoEError):
                call(s)
            assert lib.cudaPeekAtLastError() == 0, name
            layer.route(logits, bias)  # a launch that asks
    torch.cuda.synchronize()
    assert layer.device_error() == 0
