"""Dense gated feed-forward block (a shared expert beside the routed ones, or a
dense layer) over the C ABI: buffers once per problem size, forward -> y,
backward -> gradients. torch only allocates device memory and supplies the
stream; every product runs in the CUDA library.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import dense_ptr, matrix_ptr

ELT = {torch.bfloat16: _lib.MOE_ELT_BF16, torch.float16: _lib.MOE_ELT_FP16,
       torch.float32: _lib.MOE_ELT_FP32}
ACTIVATIONS = {"silu": _lib.FFN_SILU, "gelu": _lib.FFN_GELU_TANH}


def activation_code(name: str) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation {name!r}: one of {sorted(ACTIVATIONS)}")
    return ACTIVATIONS[name]


@dataclass
class FFNGrads:
    dx: torch.Tensor
    dw_gate: torch.Tensor
    dw_up: torch.Tensor
    dw_down: torch.Tensor


class GatedFFN:
    """y = (h(x Wg^T) * (x Wu^T)) Wd^T with h = "silu" or "gelu" (tanh form).

    N tokens, H hidden, I inner width (H, I multiples of 8), dtype bf16 or fp16;
    wg, wu [I, H], wd [H, I]. The buffers belong to one problem size and are
    reused by every call, so a result is valid until the next call. x and dy may
    be row-strided views (pitch a multiple of 8). training=False allocates no
    saved values and no gradients. grad_dtype: type of the weight gradients
    (dtype, or torch.float32)."""

    def __init__(self, N, H, I, dtype=torch.bfloat16, activation="silu", device="cuda",
                 training=True, grad_dtype=None, kernel=0):
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"dtype {dtype}: bfloat16 or float16")
        grad_dtype = dtype if grad_dtype is None else grad_dtype
        if grad_dtype not in (dtype, torch.float32):
            raise ValueError(f"grad_dtype {grad_dtype}: {dtype} or float32")
        self.N, self.H, self.I, self.dtype = int(N), int(H), int(I), dtype
        self.p = _lib.ffn_problem(N, H, I, ELT[dtype], activation_code(activation), ELT[grad_dtype],
                                  kernel)
        self._p = ctypes.byref(self.p)
        self._tokens, self._inner = (self.N, self.H), (self.N, self.I)
        self._w_in, self._w_out = (self.I, self.H), (self.H, self.I)
        nbytes = _lib.ffn_workspace_bytes(self.p)  # also checks the sizes
        dev = torch.device(device)
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)  # clears the error word
        self.y = torch.empty((N, H), dtype=dtype, device=dev)
        self._dev = self.y.get_device()  # -1 on the host
        self.g = self.u = self.a = self.grads = None
        if training:
            self.g, self.u, self.a = (torch.empty((N, I), dtype=dtype, device=dev) for _ in range(3))
            self.grads = FFNGrads(dx=torch.empty((N, H), dtype=dtype, device=dev),
                                  dw_gate=torch.empty((I, H), dtype=grad_dtype, device=dev),
                                  dw_up=torch.empty((I, H), dtype=grad_dtype, device=dev),
                                  dw_down=torch.empty((H, I), dtype=grad_dtype, device=dev))

    def _weights(self, wg, wu, wd):
        if self._dev < 0:  # kernels would fault on host addresses
            raise ValueError("expected a GatedFFN on a CUDA device")
        return (dense_ptr("wg", wg, self._w_in, self.dtype, self._dev),
                dense_ptr("wu", wu, self._w_in, self.dtype, self._dev),
                dense_ptr("wd", wd, self._w_out, self.dtype, self._dev))

    def _forward(self, x, wg, wu, wd, saved, stream):
        xp, ldx = matrix_ptr("x", x, self._tokens, self.dtype, self._dev)
        y = self.y
        _lib._call("ffn_forward", self._p, xp, ldx, *self._weights(wg, wu, wd), *saved, y.data_ptr(),
                   self.H, self.ws.data_ptr(), _lib.stream_on(self._dev, stream))
        return y

    def forward(self, x, wg, wu, wd, stream=None):
        """y, keeping what backward() reads in self.g, self.u and self.a."""
        if self.g is None:
            raise ValueError("forward() saves values for backward(): needs training=True "
                             "(forward_inference() does not)")
        return self._forward(x, wg, wu, wd, (self.g.data_ptr(), self.u.data_ptr(), self.a.data_ptr()),
                             stream)

    def forward_inference(self, x, wg, wu, wd, stream=None):
        """y without saved values."""
        return self._forward(x, wg, wu, wd, (None, None, None), stream)

    def backward(self, dy, x, wg, wu, wd, saved=None, stream=None) -> FFNGrads:
        """Gradients for dy. saved: the (g, u, a) of the forward when they are not
        this object's own (several micro-batches in flight)."""
        d = self.grads
        if d is None:
            raise ValueError("backward() needs training=True")
        xp, ldx = matrix_ptr("x", x, self._tokens, self.dtype, self._dev)
        dyp, lddy = matrix_ptr("dy", dy, self._tokens, self.dtype, self._dev)
        g, u, a = (self.g, self.u, self.a) if saved is None else saved
        inner, dtype, dev = self._inner, self.dtype, self._dev
        _lib._call("ffn_backward", self._p, xp, ldx, dense_ptr("g", g, inner, dtype, dev),
                   dense_ptr("u", u, inner, dtype, dev), dense_ptr("a", a, inner, dtype, dev),
                   *self._weights(wg, wu, wd), dyp, lddy, d.dx.data_ptr(), self.H, d.dw_gate.data_ptr(),
                   d.dw_up.data_ptr(), d.dw_down.data_ptr(), self.ws.data_ptr(), _lib.stream_on(self._dev, stream))
        return d

    def device_error(self, stream=None) -> int:
        return _lib.ffn_get_device_error(self.p, self.ws, stream)

    def clear_device_error(self, stream=None):
        _lib.ffn_clear_device_error(self.p, self.ws, stream)
