"""The binding of the 8-bit expert layer: operands on other devices than the current one,
of other types or forms, are refused before the library is called, and what a call makes
is its stream's memory.  On the CPU, with tensors that only have a shape."""
import pytest
import torch

import any_precision_weight_gb300 as pw
from any_precision_weight_gb300.model import F8Experts

from test_operator_devices import library  # noqa: F401
from test_operator_memory import Lib, Shape, Stream, made  # noqa: F401

F16, F32, F8, I32 = torch.float16, torch.float32, torch.float8_e4m3fn, torch.int32
T, K, N, E, k = 40, 256, 384, 8, 2
KB, NB = 2, 3


class Tensor(Shape):
    """A Shape with strides of any number of axes."""

    def __init__(self, shape, dtype, index=0, contiguous=True):
        super().__init__(shape, dtype, index, contiguous=contiguous)
        s, self.strides = 1, ()
        for n in reversed(shape):
            self.strides = (s, *self.strides)
            s *= n

    def __getitem__(self, at):
        return Tensor((*self.shape[:-1], at[-1].stop), self.dtype, self.index, False)


def t(dtype, *shape, at=0, contiguous=True):
    return Tensor(shape, dtype, at, contiguous)


def quant(**kw):
    return pw.pw_quant_f8(**{**dict(x=t(F16, T, K), rows=t(I32, T), per=2, q=t(F8, T, K), scale=t(F32, T, KB)), **kw})


def silu(**kw):
    return pw.pw_silu_quant_f8(**{**dict(x=t(F16, T, 2 * K), q=t(F8, T, K), scale=t(F32, T, KB)), **kw})


def blocks(**kw):
    return pw.pw_quant_f8_blocks(**{**dict(w=t(F16, N, K), q=t(F8, N, K), scale=t(F32, NB, KB)), **kw})


def linear(**kw):
    a = dict(x=t(F8, T, K), x_scale=t(F32, T, KB), w=t(F8, N, K), w_scale=t(F32, NB, KB), bias=t(F16, N), out=t(F16, T, N))
    return pw.pw_linear_f8(**{**a, **kw})


def grouped(**kw):
    a = dict(x=t(F8, T, K), x_scale=t(F32, T, KB), w=t(F8, E, N, K), w_scale=t(F32, E, NB, KB), offsets=t(I32, E + 1),
             bias=t(F16, E, N), out=t(F16, T, N))
    return pw.pw_grouped_linear_f8(**{**a, **kw})


def route(**kw):
    out = dict(idx=t(I32, T, k), weight=t(F32, T, k), offsets=t(I32, E + 1), perm=t(I32, T * k), inv=t(I32, T * k))
    out.update((n, kw.pop(n)) for n in list(kw) if n in out)
    return pw.pw_route(**{**dict(logits=t(F32, T, E), top_k=k), **kw}, out=pw.Routing(**out))


def combine(**kw):
    a = dict(y=t(F16, T * k, N), weight=t(F32, T, k), inv=t(I32, T * k), residual=t(F16, T, N), out=t(F16, T, N))
    return pw.pw_combine(**{**a, **kw})


WHAT = [(quant, dict(x=(F16, T, K), rows=(I32, T), q=(F8, T, K), scale=(F32, T, KB))),
        (silu, dict(x=(F16, T, 2 * K), q=(F8, T, K), scale=(F32, T, KB))),
        (blocks, dict(w=(F16, N, K), q=(F8, N, K), scale=(F32, NB, KB))),
        (linear, dict(x=(F8, T, K), x_scale=(F32, T, KB), w=(F8, N, K), w_scale=(F32, NB, KB), bias=(F16, N), out=(F16, T, N))),
        (grouped, dict(x=(F8, T, K), x_scale=(F32, T, KB), w=(F8, E, N, K), w_scale=(F32, E, NB, KB), offsets=(I32, E + 1),
                       bias=(F16, E, N), out=(F16, T, N))),
        (route, dict(logits=(F32, T, E), idx=(I32, T, k), weight=(F32, T, k), offsets=(I32, E + 1), perm=(I32, T * k),
                     inv=(I32, T * k))),
        (combine, dict(y=(F16, T * k, N), weight=(F32, T, k), inv=(I32, T * k), residual=(F16, T, N), out=(F16, T, N)))]
OPERANDS = [(f, name, what) for f, a in WHAT for name, what in a.items()]


@pytest.mark.parametrize("call,name,what", OPERANDS)
def test_an_operand_elsewhere_is_refused(call, name, what, library, monkeypatch):  # noqa: F811
    for devices, places in ((2, (1, -1)), (1, (-1,))):
        monkeypatch.setattr(pw, "_devices", devices)
        call()
        assert library.called
        for at in places:
            library.called.clear()
            with pytest.raises(ValueError):
                call(**{name: t(*what, at=at)})
            assert not library.called


@pytest.mark.parametrize("call,name,what", OPERANDS)
def test_an_operand_of_another_type_or_shape_is_refused(call, name, what, library):  # noqa: F811
    dtype, *shape = what
    call()
    library.called.clear()
    for other in ((torch.int64, *shape), (dtype, *shape[:-1], shape[-1] + 1), (dtype, *shape, 1)):
        with pytest.raises((TypeError, ValueError)):
            call(**{name: t(*other)})
        assert not library.called


@pytest.mark.parametrize("call", [f for f, _ in WHAT])
def test_another_current_device_or_stream_is_refused(call, library, monkeypatch):  # noqa: F811
    call(stream=Stream())
    library.called.clear()
    far = Stream()
    far.device_index = 1
    with pytest.raises(ValueError):
        call(stream=far)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(ValueError):
        call()
    assert not library.called


@pytest.mark.parametrize("call,n", [
    (lambda s: pw.pw_quant_f8(t(F16, T, K), stream=s), 2), (lambda s: pw.pw_silu_quant_f8(t(F16, T, K), stream=s), 2),
    (lambda s: pw.pw_quant_f8_blocks(t(F16, T, K), stream=s), 2), (lambda s: linear(out=None, stream=s), 1),
    (lambda s: grouped(out=None, stream=s), 1), (lambda s: combine(out=None, stream=s), 1),
    (lambda s: pw.pw_route(t(F32, T, E), k, stream=s), 5),
    (lambda s: F8Experts(t(F8, E, 2 * N, K), t(F8, E, K, N), t(F32, E, 6, KB), t(F32, E, KB, NB)).forward(
        t(F16, T, K), t(F32, T, E), k, True, stream=s), 12)])
def test_what_a_call_makes_is_its_streams_memory(call, n, made, monkeypatch):  # noqa: F811
    library = Lib()
    monkeypatch.setattr(pw, "lib", lambda: library)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device, e=torch.empty: t(dtype, *e(shape, dtype, device).shape))
    stream = Stream()
    call(stream)
    assert made == [stream] * n
    made.clear()
    call(None)
    assert made == [None] * n


def test_experts_refuse_weights_that_do_not_belong_together():
    with pytest.raises(ValueError):
        F8Experts(t(F8, E, 2 * N, K), t(F8, E, K, N + 1))
    with pytest.raises(ValueError):
        F8Experts(t(F8, E, 2 * N, K), t(F8, E, K, N))   # e4m3 without scales
