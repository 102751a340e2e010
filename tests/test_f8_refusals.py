"""Arguments that the operators of an 8-bit expert layer refuse, on the host: every check
comes before anything is launched, so the addresses are never used."""
import pytest
import torch

import any_precision_weight_gb300 as pw

P = 0x10000        # an aligned address that nothing reads
BIG = (1 << 30) + 1


def call(name, a, kw):
    assert set(kw) <= set(a)
    return getattr(pw.lib(), name)(*{**a, **kw}.values(), None)


def refused(name, a, kw, code=pw.PW_EINVAL):
    assert call(name, a, kw) == code
    assert name.encode() in pw.lib().pw_last_error()


QUANT = dict(x=P, ldx=200, n=4, rows=P, per=2, T=6, K=200, dt=pw.PW_F16, q=P, ldq=208, scale=P, lds=2)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=BIG), dict(K=0), dict(K=BIG, ldx=1 << 31, ldq=1 << 31, lds=1 << 24), dict(dt=3), dict(dt=-1), dict(per=0),
    dict(n=-1), dict(rows=None, n=5), dict(x=None), dict(q=None), dict(scale=None), dict(ldx=199), dict(ldq=199),
    dict(lds=1), dict(x=P + 1), dict(scale=P + 2), dict(rows=P + 2)])
def test_quant(kw):
    refused("pw_quant_f8", QUANT, kw)


SILU = dict(x=P, ldx=400, T=6, K=200, dt=pw.PW_F32, q=P, ldq=208, scale=P, lds=2)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(K=0), dict(dt=7), dict(x=None), dict(q=None), dict(scale=None), dict(ldx=399), dict(ldq=199),
    dict(lds=1), dict(x=P + 2), dict(scale=P + 1)])
def test_silu_and_blocks(kw):
    refused("pw_silu_quant_f8", SILU, kw)
    refused("pw_quant_f8_blocks", {**SILU, "ldx": 200}, {**kw, "ldx": kw["ldx"] - 200} if "ldx" in kw else kw)


LINEAR = dict(x=P, ldx=208, xs=P, ldxs=2, w=P, ldw=208, ws=P, ldws=2, bias=None, T=3, N=40, K=200, dt=pw.PW_F16, out=P,
              ldo=40)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=BIG), dict(N=0), dict(N=BIG, ldo=1 << 31), dict(K=0), dict(K=BIG, ldx=1 << 31, ldw=1 << 31, ldxs=1 << 24, ldws=1 << 24),
    dict(dt=3), dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(out=None), dict(ldx=192), dict(ldw=192),
    dict(ldx=204), dict(ldw=216), dict(ldxs=1), dict(ldws=1), dict(ldo=39), dict(x=P + 8), dict(w=P + 8), dict(xs=P + 2),
    dict(ws=P + 2), dict(out=P + 1), dict(bias=P + 1), dict(T=1 << 30, N=1 << 30, ldo=1 << 30)])
def test_linear(kw):
    refused("pw_linear_f8", LINEAR, kw)


GROUPED = dict(x=P, ldx=208, xs=P, ldxs=2, w=P, ldw=208, gw=208 * 40, ws=P, ldws=2, gws=2, off=P, bias=None, T=3, E=5, N=40,
               K=200, dt=pw.PW_F16, out=P, ldo=40)


@pytest.mark.parametrize("kw", [
    dict(off=None), dict(off=P + 2), dict(E=0), dict(E=pw.MAX_GROUPS + 1), dict(gw=208 * 40 + 8), dict(gw=-16), dict(gws=-1),
    dict(T=-1), dict(N=0), dict(K=0), dict(dt=9), dict(x=None), dict(w=None), dict(ldx=204), dict(ldw=200), dict(ldo=39),
    dict(out=P + 1), dict(bias=P + 1)])
def test_grouped(kw):
    refused("pw_grouped_linear_f8", GROUPED, kw)


ROUTE = dict(x=P, ld=60, T=4, E=60, k=4, renorm=0, idx=P, w=P, off=P, perm=P, inv=P)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(E=0, k=0), dict(E=pw.MAX_GROUPS + 1, ld=600), dict(k=0), dict(k=61), dict(T=1 << 29), dict(ld=59),
    dict(x=None), dict(idx=None), dict(w=None), dict(off=None), dict(perm=None), dict(inv=None), dict(x=P + 2),
    dict(idx=P + 1), dict(w=P + 1), dict(off=P + 1), dict(perm=P + 2), dict(inv=P + 2)])
def test_route(kw):
    refused("pw_route", ROUTE, kw)


COMBINE = dict(y=P, ldy=100, n=8, dt=pw.PW_F16, w=P, inv=P, res=None, ldr=0, T=4, k=2, H=100, odt=pw.PW_F32, out=P, ldo=100)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=BIG), dict(H=0), dict(H=BIG, ldy=1 << 31, ldo=1 << 31), dict(k=0), dict(k=pw.MAX_GROUPS + 1), dict(n=-1),
    dict(dt=3), dict(odt=3), dict(y=None), dict(w=None), dict(inv=None), dict(out=None), dict(ldy=99), dict(ldo=99),
    dict(res=P, ldr=99), dict(y=P + 1), dict(w=P + 2), dict(inv=P + 2), dict(out=P + 2), dict(res=P + 2, ldr=100)])
def test_combine(kw):
    refused("pw_combine", COMBINE, kw)


def test_no_rows_is_no_work():
    none = dict(x=None, q=None, scale=None, T=0)
    assert call("pw_quant_f8", QUANT, {**none, "rows": None, "n": 0}) == pw.PW_OK
    assert call("pw_silu_quant_f8", SILU, none) == pw.PW_OK
    assert call("pw_quant_f8_blocks", SILU, none) == pw.PW_OK
    assert call("pw_linear_f8", LINEAR, dict(T=0, x=None, w=None, out=None)) == pw.PW_OK
    assert call("pw_grouped_linear_f8", GROUPED, dict(T=0, x=None, off=None, out=None)) == pw.PW_OK
    assert call("pw_combine", COMBINE, dict(T=0, y=None, out=None)) == pw.PW_OK
    assert pw.lib().pw_linear_f8_status(None, None) == pw.PW_EINVAL


def test_binding_refuses_other_types_and_forms():
    x = torch.zeros(2, 64, dtype=torch.float16)
    q, s = torch.zeros(2, 64).to(torch.float8_e4m3fn), torch.zeros(2, 1)
    for f in (lambda: pw.pw_quant_f8(x), lambda: pw.pw_silu_quant_f8(x), lambda: pw.pw_quant_f8_blocks(x),
              lambda: pw.pw_linear_f8(q, s, q, s), lambda: pw.pw_grouped_linear_f8(q, s, q[None], s[None], s[:, 0]),
              lambda: pw.pw_route(s, 1), lambda: pw.pw_combine(x, s, s)):
        with pytest.raises(ValueError):
            f()
