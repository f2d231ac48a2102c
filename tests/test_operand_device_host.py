"""Operands of the dense block and the 4-bit formats on a GPU other than the object's,
and calls while another GPU is current, are refused before anything is launched: a
kernel would be handed addresses of another GPU. Played here with tensors that only
report where they are (no GPU)."""
import pytest
import torch

from mixture_experts_layer_schedule_gb300 import FP4Linear, FP4Tensor, GatedFFN, _lib, build

BF = torch.bfloat16


class On:
    """A dense tensor that says it is on GPU `index`."""

    def __init__(self, index, shape, dtype=BF, stride=None):
        self.index, self.shape, self.dtype = index, torch.Size(shape), dtype
        self.device, self.is_cuda = torch.device("cuda", index), True
        self._stride = stride or (shape[1], 1)

    def get_device(self):
        return self.index

    def stride(self):
        return self._stride

    def is_contiguous(self):
        return self._stride == (self.shape[1], 1)

    def data_ptr(self):
        return 4096


@pytest.fixture
def made(monkeypatch):
    """Objects are made on the host; from the first launch() on, the library's calls are
    only noted, with GPU 0 as the current one."""
    build.build()
    _lib.load()
    names = []

    def launch():
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
        monkeypatch.setattr(_lib, "_call", lambda name, *a: names.append(name))
        return names

    return launch


def ffn(dev):
    f = GatedFFN(4, 256, 128, device="cpu")
    f._dev = dev
    f.g, f.u, f.a = (On(dev, (4, 128)) for _ in range(3))
    return f


SHAPES = dict(x=(4, 256), wg=(128, 256), wu=(128, 256), wd=(256, 128), dy=(4, 256))


def test_dense_block(made):
    f, f1 = ffn(0), ffn(1)
    names = made()

    def args(dev=0, **kw):
        return {**{k: On(dev, s) for k, s in SHAPES.items()}, **kw}

    def forward(f, dy, **kw):
        return f.forward_inference(**kw)

    def backward(f, **kw):
        return f.backward(**kw)

    forward(f, **args())
    backward(f, **args())
    assert names == ["ffn_forward", "ffn_backward"]
    for name, shape in SHAPES.items():
        for call in (backward,) if name == "dy" else (forward, backward):
            with pytest.raises(ValueError, match=f"{name}: expected a tensor on cuda:0, got one on cuda:1"):
                call(f, **args(**{name: On(1, shape)}))
    with pytest.raises(ValueError, match="u: expected a tensor on cuda:0"):
        f.backward(**args(), saved=(f.g, On(1, (4, 128)), f.a))
    with pytest.raises(ValueError, match="contiguous"):
        forward(f, **args(wg=On(1, (128, 256), stride=(1, 128))))
    for call in (forward, backward):
        with pytest.raises(ValueError, match="current device is cuda:0, the buffers are on cuda:1"):
            call(f1, **args(1))
    assert len(names) == 2


def test_4_bit_forms(made):
    def weight(dev):
        w = FP4Tensor(32, 64, device="cpu")
        w._dev = dev
        return w

    def linear(dev):
        lin = FP4Linear(4, 32, 64, device="cpu")
        lin._dev = dev
        return lin

    t, t1, lin, lin1 = weight(0), weight(1), linear(0), linear(1)
    names = made()
    x, x1, src = On(0, (4, 64)), On(1, (4, 64)), On(0, (32, 64))
    t.quantize(src)
    t.dequantize(src)
    lin.forward(x, t)
    lin.forward_gated(x, t, t)
    assert names == ["fp4_quantize", "fp4_dequantize", "fp4_linear", "fp4_gated_linear"]
    for call, match in ((lambda: t.quantize(On(1, (32, 64))), "src: expected a tensor on cuda:0"),
                        (lambda: t.dequantize(On(1, (32, 64))), "out: expected a tensor on cuda:0"),
                        (lambda: lin.forward(x1, t), "x: expected a tensor on cuda:0"),
                        (lambda: lin.forward(x, t1), "weights on cuda:1: expected them on cuda:0"),
                        (lambda: lin.forward_gated(x, t, t1), "weights on cuda:1"),
                        (lambda: t1.quantize(On(1, (32, 64))), "current device is cuda:0"),
                        (lambda: t1.dequantize(On(1, (32, 64))), "current device is cuda:0"),
                        (lambda: lin1.forward(x1, t1), "current device is cuda:0"),
                        (lambda: lin1.forward_gated(x1, t1, t1), "current device is cuda:0")):
        with pytest.raises(ValueError, match=match):
            call()
    assert len(names) == 4


def test_buffers_on_the_host_are_refused():
    build.build()
    t = FP4Tensor(32, 64, device="cpu")
    for src in (On(0, (32, 64)), torch.zeros((32, 64), dtype=BF)):
        with pytest.raises(ValueError, match="expected an FP4Tensor on a CUDA device"):
            t.quantize(src)
    with pytest.raises(ValueError, match="expected a GatedFFN on a CUDA device"):
        GatedFFN(4, 256, 128, device="cpu").forward_inference(*(On(0, SHAPES[k]) for k in ("x", "wg", "wu", "wd")))
