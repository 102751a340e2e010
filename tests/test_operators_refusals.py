"""Arguments that the operators around the layer refuse, on the host: every
check comes before anything is launched, so the addresses are never used."""
import pytest

import any_precision_weight_gb300 as pw

P = 0x10000        # an aligned address that nothing reads


def _norm(**kw):
    a = dict(x=P, ldx=64, r=None, ldr=0, w=P, eps=1e-6, T=2, H=64, dt=pw.PW_F16, sum=None, lds=0, y=P, ldy=64,
             q=None, ldq=0, scale=None)
    a.update(kw)
    return pw.lib().pw_rms_norm(*[a[k] for k in ("x", "ldx", "r", "ldr", "w", "eps", "T", "H", "dt", "sum", "lds",
                                                  "y", "ldy", "q", "ldq", "scale")], None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(dt=3), dict(dt=-1), dict(eps=-1e-6), dict(eps=float("nan")), dict(x=None),
    dict(w=None), dict(y=None), dict(q=P, ldq=64), dict(ldx=63), dict(r=P, ldr=63), dict(sum=P, lds=63),
    dict(ldy=63), dict(q=P, ldq=63, scale=P), dict(x=P + 1), dict(dt=pw.PW_F32, y=P + 2), dict(w=P + 1),
    dict(q=P, ldq=64, scale=P + 2), dict(H=(1 << 30) + 1, ldx=1 << 31, ldy=1 << 31)])
def test_norm_refuses(kw):
    assert _norm(**kw) == pw.PW_EINVAL
    assert b"pw_rms_norm" in pw.lib().pw_last_error()


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(K=0), dict(dt=9), dict(x=None), dict(q=None), dict(scale=None), dict(ldx=31), dict(ldq=31),
    dict(x=P + 1), dict(scale=P + 1), dict(K=(1 << 30) + 1, ldx=1 << 31, ldq=1 << 31)])
def test_quant_refuses(kw):
    a = dict(x=P, ldx=32, T=2, K=32, dt=pw.PW_F16, q=P, ldq=32, scale=P)
    a.update(kw)
    assert pw.lib().pw_quant_i8(*[a[k] for k in ("x", "ldx", "T", "K", "dt", "q", "ldq", "scale")],
                                None) == pw.PW_EINVAL
    assert b"pw_quant_i8" in pw.lib().pw_last_error()


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(N=0), dict(K=0), dict(K=pw.MAX_K_I8 + 1, ldx=1 << 20, ldw=1 << 20), dict(dt=3), dict(x=None),
    dict(xs=None), dict(w=None), dict(ws=None), dict(out=None), dict(ldx=48), dict(ldw=48), dict(ldo=7),
    dict(x=P + 8), dict(w=P + 8), dict(ldx=72), dict(ldw=72), dict(out=P + 1), dict(bias=P + 1), dict(xs=P + 2),
    dict(ws=P + 1), dict(N=(1 << 30) + 1, ldo=1 << 31), dict(T=(1 << 30) + 1, sp=P, sb=1 << 62)])
def test_linear_refuses(kw):
    assert _linear(**kw) == pw.PW_EINVAL
    assert b"pw_linear_i8" in pw.lib().pw_last_error()


def _linear(**kw):
    a = dict(x=P, ldx=64, xs=P, w=P, ldw=64, ws=P, bias=None, T=2, N=8, K=64, dt=pw.PW_F16, out=P, ldo=8, sp=None,
             sb=0)
    a.update(kw)
    return pw.lib().pw_linear_i8(*[a[k] for k in ("x", "ldx", "xs", "w", "ldw", "ws", "bias", "T", "N", "K", "dt",
                                                   "out", "ldo", "sp", "sb")], None)


def test_linear_workspace():
    assert pw.pw_linear_i8_workspace_bytes(16, 4096) == 0
    assert pw.pw_linear_i8_workspace_bytes(17, 100) == 17 * 128 * 2
    assert pw.pw_linear_i8_workspace_bytes(-1, 100) == 0 and pw.pw_linear_i8_workspace_bytes(4, 0) == 0
    assert _linear(T=17) == pw.PW_ENOMEM
    assert _linear(T=17, sp=P, sb=17 * 128 - 1) == pw.PW_ENOMEM
    assert _linear(T=17, sp=None, sb=1 << 20) == pw.PW_ENOMEM
    assert _linear(T=17, sp=P + 16, sb=1 << 20) == pw.PW_EINVAL


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(V=0), dict(V=(1 << 30) + 1, ld=1 << 31), dict(dt=3), dict(top=-1), dict(top=pw.MAX_TOP + 1), dict(V=4, ld=4, top=5), dict(x=None),
    dict(ld=99), dict(ids=None), dict(tl=None), dict(ti=None), dict(x=P + 1), dict(ids=P + 4, ids64=1),
    dict(ids=P + 2), dict(lp=P + 1), dict(rank=P + 2), dict(ent=P + 1), dict(ti=P + 2), dict(tl=P + 2)])
def test_logprobs_refuses(kw):
    a = dict(x=P, ld=100, dt=pw.PW_F16, T=2, V=100, ids=P, ids64=0, top=3, lp=P, rank=P, ent=P, ti=P, tl=P)
    a.update(kw)
    assert pw.lib().pw_logprobs(*[a[k] for k in ("x", "ld", "dt", "T", "V", "ids", "ids64", "top", "lp", "rank",
                                                  "ent", "ti", "tl")], None) == pw.PW_EINVAL
    assert b"pw_logprobs" in pw.lib().pw_last_error()


def test_no_rows_is_no_work():
    assert _norm(T=0, x=None, y=None, w=None) == pw.PW_OK
    L = pw.lib()
    assert L.pw_quant_i8(None, 32, 0, 32, pw.PW_F16, None, 32, None, None) == pw.PW_OK
    assert _linear(T=0, x=None, w=None) == pw.PW_OK
    assert L.pw_logprobs(None, 100, pw.PW_F16, 0, 100, None, 0, 0, None, None, None, None, None, None) == pw.PW_OK


def test_binding_refuses_tensors_off_the_gpu():
    import torch
    x = torch.zeros(2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        pw.pw_rms_norm(x, x[0])
    with pytest.raises(ValueError):
        pw.pw_quant_i8(x)
    with pytest.raises(ValueError):
        pw.pw_logprobs(x)
    i = torch.zeros(2, 64, dtype=torch.int8)
    with pytest.raises(ValueError):
        pw.pw_linear_i8(i, x[:, 0].float(), i, x[:, 0].float())
