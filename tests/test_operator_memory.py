"""Whose memory the layer's and the operators' outputs and workspaces are: with `stream` given they
come from that stream's pool, since a block freed on another stream may still be
in use by work queued there.  On the CPU, with tensors that only have a shape."""
import contextlib

import pytest
import torch

import any_precision_weight_gb300 as pw

DEV = torch.device("cuda", 0)


class Shape:
    """What the binding asks of a CUDA tensor, without memory."""

    def __init__(self, shape, dtype, index=0, ld=None, contiguous=True):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.device = torch.device("cuda", index) if index >= 0 else torch.device("cpu")
        self.index, self.is_cuda, self.contiguous = index, index >= 0, contiguous
        self.strides = (ld or self.shape[-1], 1)[-len(shape):]

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self.strides

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return self.shape.numel()

    def __getitem__(self, at):
        return Shape((self.shape[0], at[1].stop), self.dtype, self.index, self.shape[1], False)


class Stream:
    cuda_stream = 99
    device_index = 0
    device = DEV


class Lib:
    """A library whose calls all succeed."""

    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        if name == "pw_linear_i8_workspace_bytes":
            return lambda T, K: 2 * T * K if T > 16 else 0
        return lambda *a: self.called.append(name) or 0


@pytest.fixture
def made(monkeypatch):
    """The streams whose memory the calls allocate, in order (None: the current one)."""
    streams, current = [], [None]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(shape, dtype, device):
        streams.append(current[-1])
        return Shape((shape,) if isinstance(shape, int) else shape, dtype)

    library = Lib()
    monkeypatch.setattr(pw, "lib", lambda: library)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return streams


X = Shape((40, 64), torch.float16)
Q, S = Shape((40, 64), torch.int8), Shape((40,), torch.float32)
W = Shape((64,), torch.float16)
IDS = Shape((40,), torch.int64)
# a call and how many tensors it makes
CALLS = [(lambda s: pw.pw_rms_norm(X, W, stream=s), 1), (lambda s: pw.pw_rms_norm(X, W, residual=X, stream=s), 2),
         (lambda s: pw.pw_rms_norm_i8(X, W, stream=s), 2), (lambda s: pw.pw_rms_norm_i8(X, W, residual=X, stream=s), 3),
         (lambda s: pw.pw_quant_i8(X, stream=s), 2), (lambda s: pw.pw_linear_i8(Q, S, Q, S, stream=s), 2),
         (lambda s: pw.pw_logprobs(X, stream=s), 3), (lambda s: pw.pw_logprobs(X, IDS, top=4, stream=s), 5)]


@pytest.mark.parametrize("call,n", CALLS)
def test_what_a_call_makes_is_its_streams_memory(call, n, made):
    stream = Stream()
    call(stream)
    assert made == [stream] * n
    made.clear()
    call(None)
    assert made == [None] * n


@pytest.fixture
def layer(made, monkeypatch):
    monkeypatch.setattr(torch, "empty_like", lambda x: torch.empty(x.shape, x.dtype, x.device))
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    m = object.__new__(pw.PagedMoE)
    m.L, m.E, m.H, m.I, m.device, m.guards, m._t = 1, 8, 64, 128, DEV, None, None
    return m


LOGITS = Shape((40, 8), torch.float32)
FORWARDS = [(lambda m, s: m.pw_moe_forward(0, X, LOGITS, 2, True, stream=s), 2),
            (lambda m, s: m.pw_moe_forward(0, X, LOGITS, 2, True, routing=True, stream=s), 6),
            (lambda m, s: m.pw_moe_forward_host(0, X, LOGITS, 2, True, X, stream=s), 1),
            (lambda m, s: m.pw_moe_forward_noalloc(0, X, LOGITS, 2, True, stream=s), 1)]


@pytest.mark.parametrize("call,n", FORWARDS)
def test_what_a_forward_makes_is_its_streams_memory(call, n, layer, made):
    stream = Stream()
    call(layer, stream)
    assert made == [stream] * n
    made.clear()
    call(layer, None)
    assert made == [None] * n
