"""4-bit block formats (MXFP4, NVFP4) over the C ABI: quantised matrices and
products with 4-bit weights. torch only allocates device memory and supplies
the stream; quantiser, read-back and products run in the CUDA library.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import matrix_ptr
from .ffn import ELT, activation_code

FORMATS = {"mxfp4": _lib.FP4_MX, "nvfp4": _lib.FP4_NV}


def _format(name):
    if name not in FORMATS:
        raise ValueError(f"format {name!r}: one of {sorted(FORMATS)}")
    return FORMATS[name]


def _elt(t):
    if t.dtype not in ELT:
        raise ValueError(f"dtype {t.dtype}: one of {[str(d) for d in ELT]}")
    return ELT[t.dtype]


class FP4Tensor:
    """A [rows, cols] matrix in 4 bits (cols a multiple of 32): packed codes q,
    block scales s in the order the products read, and the tensor scale (NVFP4;
    1 for MXFP4) that quantize() and every reader apply. All three may be set, to
    another scale or to stored codes and scales of the same sizes; every later
    call uses them."""

    def __init__(self, rows, cols, format="nvfp4", scale=1.0, device="cuda"):
        self.rows, self.cols, self.format = int(rows), int(cols), _format(format)
        n = _lib.fp4_scale_bytes(self.format, rows, cols)  # also checks the sizes
        dev = torch.device(device)
        self._q = torch.empty((self.rows, self.cols // 2), dtype=torch.uint8, device=dev)
        self._s = torch.empty(n, dtype=torch.uint8, device=dev)
        # what the library is handed; the setters below keep it in step
        self.operand = _lib.FP4Operand(self._q.data_ptr(), self._s.data_ptr(), 1.0)
        self.scale = scale
        self._shape, self._operand = (self.rows, self.cols), ctypes.byref(self.operand)
        self._dev = self._q.get_device()  # -1 on the host

    @property
    def scale(self) -> float:
        return self._scale

    @scale.setter
    def scale(self, value):
        self._scale = self.operand.scale = float(value)

    @property
    def q(self) -> torch.Tensor:
        return self._q

    @q.setter
    def q(self, t):
        self.operand.q = self._buffer("q", t, self._q)
        self._q = t

    @property
    def s(self) -> torch.Tensor:
        return self._s

    @s.setter
    def s(self, t):
        self.operand.s = self._buffer("s", t, self._s)
        self._s = t

    @staticmethod
    def _buffer(name, t, old):
        if t.device != old.device:
            raise ValueError(f"{name}: expected a tensor on {old.device}, got one on {t.device}")
        if t.shape != old.shape or t.dtype != old.dtype or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous {old.dtype} of shape {tuple(old.shape)}, got {t.dtype} "
                             f"of shape {tuple(t.shape)}")
        return t.data_ptr()

    @classmethod
    def of_weight(cls, w, format="nvfp4", stream=None) -> "FP4Tensor":
        """w [rows, cols] quantised, for NVFP4 with the power of two as tensor scale
        that puts the largest magnitude at the top of both levels (6 * 448) or
        just below: reads that magnitude on the host, so call it at load time.
        Everything runs on `stream`, and the result's memory belongs to it, as that
        of a tensor made under torch.cuda.stream(stream)."""
        with _lib.stream_scope(stream):
            scale = 1.0
            if _format(format) == _lib.FP4_NV:
                top = float(w.abs().max()) if w.numel() else 0.0
                if 0.0 < top < math.inf:
                    scale = 2.0 ** min(60, max(-60, math.ceil(math.log2(top / (6.0 * 448.0)))))
            return cls(*w.shape, format=format, scale=scale, device=w.device).quantize(w)

    def on_device(self):
        """Raises unless the buffers are on the GPU (kernels would fault on host addresses)."""
        if self._dev < 0:
            raise ValueError("expected an FP4Tensor on a CUDA device")

    def quantize(self, src, stream=None) -> "FP4Tensor":
        """Codes and scales of src (bf16, fp16 or fp32; rows may be strided)."""
        elt = _elt(src)
        sp, ld = matrix_ptr("src", src, self._shape, src.dtype, self._dev)
        self.on_device()
        _lib._call("fp4_quantize", sp, elt, self.rows, self.cols, ld, self.format, self.scale,
                   self.operand.q, self.operand.s, _lib.stream_on(self._dev, stream))
        return self

    def dequantize(self, out=None, dtype=torch.bfloat16, stream=None):
        """The values the codes stand for, rounded once to out's type. Without out, the
        memory is taken on `stream` (as under torch.cuda.stream(stream))."""
        if out is None:
            with _lib.stream_scope(stream):
                out = torch.empty((self.rows, self.cols), dtype=dtype, device=self.q.device)
        elt = _elt(out)
        op, ld = matrix_ptr("out", out, self._shape, out.dtype, self._dev)
        self.on_device()
        _lib._call("fp4_dequantize", self.operand.q, self.operand.s, self.format, self.scale, self.rows,
                   self.cols, op, elt, ld, _lib.stream_on(self._dev, stream))
        return out


class FP4Linear:
    """Products of M rows of K 16-bit activations with 4-bit weights of N
    features (FP4Tensor(N, K)), the activations quantised in the call with
    tensor scale x_scale. The buffers belong to one problem size: a result is
    valid until the next call."""

    def __init__(self, M, N, K, format="nvfp4", dtype=torch.bfloat16, activation="silu", x_scale=1.0,
                 device="cuda", kernel=0):
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"dtype {dtype}: bfloat16 or float16")
        self.M, self.N, self.K, self.dtype, self.x_scale = int(M), int(N), int(K), dtype, float(x_scale)
        self.format = _format(format)
        self.p = _lib.fp4_problem(M, N, K, self.format, ELT[dtype], activation_code(activation), kernel)
        self._p, self._x_shape, self._w_shape = ctypes.byref(self.p), (self.M, self.K), (self.N, self.K)
        nbytes = _lib.fp4_workspace_bytes(self.p)  # also checks the sizes
        dev = torch.device(device)
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        self.ws[:256].zero_()  # clears the device error word
        self.y = torch.empty((self.M, self.N), dtype=dtype, device=dev)
        self._dev = self.y.get_device()  # -1 on the host

    def _weight(self, w):
        if self._dev < 0:
            raise ValueError("expected an FP4Linear on a CUDA device")
        if w._shape != self._w_shape or w.format != self.format:
            raise ValueError(f"weights [{w.rows}, {w.cols}] of format {w.format}: expected "
                             f"[{self.N}, {self.K}] of format {self.format}")
        if w._dev != self._dev:
            w.on_device()
            raise ValueError(f"weights on cuda:{w._dev}: expected them on cuda:{self._dev}")
        return w._operand

    def forward(self, x, w: FP4Tensor, stream=None):
        """x w^T."""
        xp, ldx = matrix_ptr("x", x, self._x_shape, self.dtype, self._dev)
        _lib._call("fp4_linear", self._p, xp, ldx, self.x_scale, self._weight(w), self.y.data_ptr(),
                   self.N, self.ws.data_ptr(), _lib.stream_on(self._dev, stream))
        return self.y

    def forward_gated(self, x, w_gate: FP4Tensor, w_up: FP4Tensor, stream=None):
        """h(x w_gate^T) * (x w_up^T), h the activation."""
        xp, ldx = matrix_ptr("x", x, self._x_shape, self.dtype, self._dev)
        _lib._call("fp4_gated_linear", self._p, xp, ldx, self.x_scale, self._weight(w_gate),
                   self._weight(w_up), self.y.data_ptr(), self.N, self.ws.data_ptr(),
                   _lib.stream_on(self._dev, stream))
        return self.y

    def device_error(self, stream=None) -> int:
        return _lib.fp4_get_device_error(self.p, self.ws, stream)

    def clear_device_error(self, stream=None):
        _lib.fp4_clear_device_error(self.p, self.ws, stream)


class FP4GatedFFN:
    """The gated feed-forward block of GatedFFN with 4-bit weights, for serving:
    the gated product, then the down product, each quantising its input in the
    call. Two launches for few tokens (up to 32 at 4096 x 1536); with more tokens, or
    wider or deeper weights, a product's input is quantised by a launch of its own where
    that is expected to be faster.

    x_scale and act_scale are the NVFP4 tensor scales of x and of the inner
    activations. At 1 a block of 16 values whose largest magnitude is at most
    6 * 2^-10 becomes zeros, and below 6 * 2^-6 its scale keeps three bits or fewer;
    a power of two near max|x| / (6 * 448) uses the format's whole range."""

    def __init__(self, N, H, I, format="nvfp4", dtype=torch.bfloat16, activation="silu", device="cuda",
                 x_scale=1.0, act_scale=1.0):
        self.gate_up = FP4Linear(N, I, H, format=format, dtype=dtype, activation=activation, x_scale=x_scale,
                                 device=device)
        self.down = FP4Linear(N, H, I, format=format, dtype=dtype, x_scale=act_scale, device=device)

    @staticmethod
    def quantize_weights(wg, wu, wd, format="nvfp4"):
        """(wg, wu, wd) as FP4Tensors (done once, at load time)."""
        return tuple(FP4Tensor.of_weight(w, format) for w in (wg, wu, wd))

    def forward(self, x, wg: FP4Tensor, wu: FP4Tensor, wd: FP4Tensor, stream=None):
        return self.down.forward(self.gate_up.forward_gated(x, wg, wu, stream), wd, stream)

    def device_error(self, stream=None) -> int:
        return self.gate_up.device_error(stream) or self.down.device_error(stream)

    def clear_device_error(self, stream=None):
        self.gate_up.clear_device_error(stream)
        self.down.clear_device_error(stream)
