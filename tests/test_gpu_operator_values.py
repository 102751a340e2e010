"""The operators' outputs against the fp64 oracle by a comparison that a NaN cannot
pass: norms with what the int8 call writes beside its rows, 16-bit products, and
the norms and products of a decode step.  Tolerances as in test_gpu_operators.py."""
import itertools

import numpy as np
import pytest
import torch

import any_precision_weight_gb300 as pw
from oracle import operators as ops

from _close import assert_values
from test_gpu_decode_step import _model
from test_gpu_operators import DT, NORMS, U, _linear_case, check_q, f64, gen, place

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", NORMS + [(305, 8), (700, 256), (999, 513), (457, 4096), (310, 8191), (305, 14336)])
def test_norms_and_what_they_write_beside(T, H):
    for dt, res in itertools.product(["f16", "bf16", "f32"], [False, True]):
        rng = gen(T, H, dt, res, "values")
        x = place(rng.standard_normal((T, H), np.float32) * 2, DT[dt])
        w = torch.as_tensor(rng.normal(1, 0.3, H)).to(DT[dt]).cuda()
        r = place(rng.standard_normal((T, H), np.float32) * 3, DT[dt]) if res else None
        s, y = ops.rms_norm(f64(x), f64(w), 1e-5, f64(r) if res else None)
        # the sum's own rounding moves elements beside which it is large
        extra = np.abs(f64(w)) * 4 * U if res else 0.0
        a = pw.pw_rms_norm(x, w, 1e-5, residual=r)
        out = torch.full_like(x, float("nan"))
        b = pw.pw_rms_norm_i8(x, w, 1e-5, residual=r, out=out)
        assert_values(f64(a[0] if res else a), y, dt, 64 * U, extra)
        assert_values(f64(out), y, dt, 64 * U, extra)
        check_q(b[0], b[1], y, 72 * U)
        if res:
            assert_values(f64(a[1]), s, dt, U)
            assert_values(f64(b[2]), s, dt, U)


@pytest.mark.parametrize("T,N,K", [(1, 60, 2048), (12, 333, 1411), (24, 20001, 512), (37, 333, 4096), (100, 1411, 1411),
                                   (128, 20001, 1040), (300, 1000, 3000)])
def test_products(T, N, K):
    for dt in ("f16", "bf16", "f32"):
        x, xs, w, ws, b = _linear_case(T, N, K, dt, True, seed=1)
        out = torch.full((T, N), float("nan"), dtype=DT[dt], device="cuda")
        pw.pw_linear_i8(x, xs, w, ws, bias=b, out=out)
        acc, ref = ops.linear_i8(f64(x), f64(xs), f64(w), f64(ws), f64(b))
        prod = np.abs(acc * f64(xs)[:, None] * f64(ws)[None, :])
        if dt == "f16":   # beyond its range there is nothing to compare
            far = np.abs(ref) > 65504.0
            ref[far], prod[far] = 0.0, 0.0
            out[torch.as_tensor(far).cuda()] = 0.0
        assert_values(f64(out), ref, dt, U, extra=prod * 3 * U)


@pytest.mark.parametrize("batch", [1, 20, 100])
def test_the_norms_and_products_of_a_step(batch):
    _, m, x, ids = _model(batch)
    trace = []
    m.step(x, ids, trace=trace)
    n = 0
    for t in trace:
        if t[0] == "norm":
            _, d, r, w, y, q, s, new = t
            sr, yr = ops.rms_norm(f64(d), f64(w), 1e-6, f64(r))
            assert_values(f64(new), sr, "f16", U)
            if y is not None:
                assert_values(f64(y), yr, "f16", 64 * U, extra=8 * U)
        elif t[0] == "linear":
            _, q, s, (w, ws), out = t
            acc, ref = ops.linear_i8(f64(q), f64(s), f64(w), f64(ws))
            assert_values(f64(out), ref, "f32" if out.dtype == torch.float32 else "f16", 4 * U)
        else:
            continue
        n += 1
    assert n == 10
