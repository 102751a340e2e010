"""Operands on other devices than the current one: the library launches on the
current device, so the binding refuses them before it calls the library.  On the
CPU, with tensors that only have a shape and a device index."""
import pytest
import torch

import any_precision_weight_gb300 as pw

from test_operator_memory import Lib, Shape, Stream

F16, F32, I8, I32 = torch.float16, torch.float32, torch.int8, torch.int32
T, K, N, V = 20, 64, 32, 100


def t(dtype, *shape, at=0, contiguous=True):
    return Shape(shape, dtype, at, contiguous=contiguous)


def norm(**kw):
    a = dict(x=t(F16, T, K), weight=t(F16, K), residual=t(F16, T, K), out=t(F16, T, K), sum_out=t(F16, T, K))
    return pw.pw_rms_norm(**{**a, **kw})


def norm_i8(**kw):
    a = dict(x=t(F16, T, K), weight=t(F16, K), q=t(I8, T, K), scale=t(F32, T))
    return pw.pw_rms_norm_i8(**{**a, **kw})


def quant(**kw):
    return pw.pw_quant_i8(**{**dict(x=t(F16, T, K), q=t(I8, T, K), scale=t(F32, T)), **kw})


def linear(**kw):
    a = dict(x=t(I8, T, K), x_scale=t(F32, T), w=t(I8, N, K), w_scale=t(F32, N), bias=t(F16, N), out=t(F16, T, N),
             ws=t(torch.uint8, 1 << 20))
    return pw.pw_linear_i8(**{**a, **kw})


def logprobs(**kw):
    a = dict(logits=t(F16, T, V), ids=t(I32, T), top=3)
    out = dict(logprob=t(F32, T), rank=t(I32, T), entropy=t(F32, T), top_ids=t(I32, T, 3), top_logprobs=t(F32, T, 3))
    out.update((k, kw.pop(k)) for k in list(kw) if k in out)
    return pw.pw_logprobs(**{**a, **kw}, out=pw.LogProbs(**out))


OPERANDS = ([(norm, k, v) for k, v in dict(x=(F16, T, K), weight=(F16, K), residual=(F16, T, K), out=(F16, T, K),
                                           sum_out=(F16, T, K)).items()]
            + [(norm_i8, k, v) for k, v in dict(q=(I8, T, K), scale=(F32, T)).items()]
            + [(quant, k, v) for k, v in dict(x=(F16, T, K), q=(I8, T, K), scale=(F32, T)).items()]
            + [(linear, k, v) for k, v in dict(x=(I8, T, K), x_scale=(F32, T), w=(I8, N, K), w_scale=(F32, N), bias=(F16, N),
                                               out=(F16, T, N), ws=(torch.uint8, 1 << 20)).items()]
            + [(logprobs, k, v) for k, v in dict(logits=(F16, T, V), ids=(I32, T), logprob=(F32, T), rank=(I32, T),
                                                 entropy=(F32, T), top_ids=(I32, T, 3), top_logprobs=(F32, T, 3)).items()])


@pytest.fixture
def library(monkeypatch):
    lib = Lib()
    monkeypatch.setattr(pw, "lib", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    pw._torch()
    monkeypatch.setattr(pw, "_devices", 2)
    return lib


@pytest.mark.parametrize("call,name,what", OPERANDS)
def test_an_operand_on_the_host_is_refused_where_there_is_one_gpu(call, name, what, library, monkeypatch):
    monkeypatch.setattr(pw, "_devices", 1)
    call()
    assert library.called
    library.called.clear()
    with pytest.raises(ValueError):
        call(**{name: t(*what, at=-1)})
    assert not library.called


@pytest.mark.parametrize("at", [1, -1])
@pytest.mark.parametrize("call,name,what", OPERANDS)
def test_an_operand_elsewhere_is_refused(call, name, what, at, library):
    call()
    assert library.called
    library.called.clear()
    with pytest.raises(ValueError):
        call(**{name: t(*what, at=at)})
    assert not library.called


@pytest.mark.parametrize("call", [norm, norm_i8, quant, linear, logprobs])
def test_another_current_device_or_stream_is_refused(call, library, monkeypatch):
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


@pytest.mark.parametrize("ws", [t(F32, 1 << 18), t(torch.uint8, 1 << 20, contiguous=False)])
def test_a_workspace_of_another_form_is_refused(ws, library):
    with pytest.raises(ValueError):
        linear(ws=ws)
    assert not library.called


@pytest.mark.parametrize("name", ["top_ids", "top_logprobs"])
def test_alternatives_without_their_outputs_are_refused(name, library):
    with pytest.raises(ValueError):
        logprobs(**{name: None})
    assert not library.called
