"""Ways of working out a product in 8 bits that the test hook refuses, on the host."""
import pytest
import torch

import any_precision_weight_gb300 as pw

from test_f8_refusals import GROUPED, P, refused

WAY = dict(ctas=1, rows=128, channels=256, parts=1)


@pytest.mark.parametrize("kw", [
    dict(ctas=3), dict(ctas=-1), dict(rows=0), dict(rows=8), dict(rows=48), dict(rows=256), dict(channels=0), dict(channels=32),
    dict(channels=96), dict(channels=320), dict(parts=0), dict(parts=2), dict(parts=3), dict(parts=8), dict(ctas=2, rows=64),
    dict(ctas=0, rows=32, channels=1), dict(ctas=0, rows=8, channels=0), dict(ctas=0, rows=8, channels=65535 // 5 + 1),
    dict(ctas=0, rows=8, channels=1, parts=4), dict(off=None), dict(E=0), dict(w=None), dict(ldx=204), dict(out=P + 1)])
def test_refused(kw):
    refused("pw_debug_linear_f8", {**WAY, **GROUPED}, kw)


@pytest.mark.parametrize("kw", [dict(parts=4), dict(parts=8, K=8000), dict(ctas=2, parts=2), dict(ctas=0, rows=16, channels=1, parts=16),
                                dict(parts=2, K=8000, T=1 << 20, N=1 << 13), dict(parts=4, K=8000, ctas=2, T=1 << 23, N=600)])
def test_refused_without_groups(kw):
    one = {**WAY, **GROUPED, "off": None, "E": 1}   # K = 200: two blocks
    one["ldo"] = max(one["ldo"], kw.get("N", 0))
    wide = dict(ldx=8000, ldw=8000, ldxs=63, ldws=63) if "K" in kw else {}
    refused("pw_debug_linear_f8", one, {**kw, **wide})


def test_binding_refuses_a_tensor_off_the_gpu():
    q, s = torch.zeros(2, 64).to(torch.float8_e4m3fn), torch.zeros(2, 1)
    with pytest.raises(ValueError):
        pw.pw_debug_linear_f8((1, 128, 64, 1), q, s, q[None], s[None, :1])
