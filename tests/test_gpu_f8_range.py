"""The quantisers at the ends of the range, each value where nothing larger hides it.

Tolerances.  U = 2^-24, V = 2^-149 (fp32's last subnormal).
 * silu(g) * u: the exponential is off by 4 U and by its argument's error: |g| U for the rounding of
   g log2 e and 0.23 |g| U for that of the constant, of which the sigmoid keeps 1 - sigmoid(g).  The
   sum is off by U, the reciprocal by 2 U (or V, among the subnormals, of a sigmoid of 1 / (1 + e^-g)),
   two products by U each: e = (10 + 1.25 |g| (1 - sigmoid(g))) U + V (1 + e^-g), with what is of
   second order.  Of a block of one gate every element and the largest have the same bound: scales
   e + 2 U, quotients half a step and (2.2 e + 4 U) of themselves.
 * scales are rounded to fp32: by U, or V / 2 where they are subnormal.
"""
import numpy as np
import pytest
import torch

import any_precision_weight_gb300 as pw
from oracle import f8

from test_gpu_f8 import INF, cuda
from test_gpu_operators import DT, U, f64, gen

pytestmark = pytest.mark.gpu
V = 2.0 ** -149


def half_step(v):
    return np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10)


# gates and the size of `up` that keeps the product among the type's, and the scale among fp32's, normal numbers
GATES = [(-3.0, 1.0), (-20.0, 1.0), (-40.0, 1e4), (-60.0, 6e4), (-80.0, 6e4), (-86.5, 6e4), (-87.5, 6e4), (-88.0, 6e4), (-88.6, 6e4),
         (0.0, 1.0), (1e-4, 100.0), (1.0, 1.0), (20.0, 1.0), (88.0, 1.0), (100.0, 1.0), (6e4, 1e-3)]


@pytest.mark.parametrize("K", [128, 300, 77])
def test_silu_of_one_gate_to_a_row(K):
    for dt in DT:
        far = [] if dt == "f16" else [(1e38, 1e-3), (-88.5, 1e30), (-87.0, 1e35)]
        rng = gen(K, dt, "gates")
        rows = GATES + far
        g = np.array([[a] * K for a, _ in rows])
        u = np.array([[b] * K for _, b in rows]) * rng.uniform(-1, 1, (len(rows), K))
        x = cuda(np.concatenate([g, u], axis=1), DT[dt])
        q, s = pw.pw_silu_quant_f8(x)
        g = f64(x)[:, :1]
        assert (np.abs(g) < 88.72).sum() == len(rows) - (g > 88.72).sum()
        e = (10 + 1.25 * np.abs(g) / (1 + np.exp(np.minimum(g, 700)))) * U + V * (1 + np.exp(-g))
        assert (e < 1e-4).all()
        v, ref = f8.quotients(f8.silu_up(f64(x)))
        assert (np.abs(f64(s) - ref) <= ref * (e + 2 * U) + V / 2).all()
        assert (np.abs(f64(q) - v) <= half_step(v) * (1 + 2.2 * e) + np.abs(v) * (2.2 * e + 4 * U)).all()


def test_silu_of_gates_whose_exponential_is_infinite():
    for dt in DT:
        top = {"f16": 6e4, "bf16": 1e38, "f32": 1e38}[dt]
        g = np.array([[a] * 150 for a in (-89.0, -100.0, -1000.0, -top)])
        x = cuda(np.concatenate([g, np.full_like(g, top)], axis=1), DT[dt])
        q, s = pw.pw_silu_quant_f8(x)
        assert (f64(s) == 0).all() and (f64(q) == 0).all()


# powers that make the largest of a block 448 of them: quotients are small whole numbers and halves
@pytest.mark.parametrize("power", [-98, -101, -108, -109, -110, -126, -130, -133, -140, -149])
def test_ties_of_tiny_blocks(power):
    """448 / max past fp32's range, and blocks of subnormals: halves go to the even number."""
    n = np.array([448, 17, 19, 21, 23, 34, 38, 9, 11, -17, -19, 1, -1, 0, 25, 27, 272, 304, 400, 416, 432, -432, 240, 248])
    for dt in ("bf16", "f32"):
        if dt == "bf16" and power < -133:
            continue
        x = cuda(n[None] * 2.0 ** power, DT[dt])
        assert np.array_equal(f64(x), n[None] * 2.0 ** power)
        for got, s in (pw.pw_quant_f8(x), pw.pw_quant_f8_blocks(x)):
            assert np.array_equal(f64(got), f8.e4m3(n[None])) and (f64(s) == 2.0 ** power).all()


@pytest.mark.parametrize("power", [-99, -100, -104, -112, -118, -124])
def test_numbers_of_tiny_blocks(power):
    for dt in ("bf16", "f32"):
        rng = gen(-power, dt, "tiny")
        x = cuda(rng.normal(0, 1, (40, 300)) * 2.0 ** power, DT[dt])
        for (q, s), rows in ((pw.pw_quant_f8(x), 1), (pw.pw_quant_f8_blocks(x), 128)):
            v, ref = f8.quotients(f64(x), rows)
            assert (np.abs(f64(s) - ref) <= ref * U + V / 2).all()
            want = f8.e4m3(v)
            if dt == "bf16":
                assert np.array_equal(f64(q), want)
            else:
                assert (np.abs(f64(q) - v) <= np.abs(want - v) + 2 * U * np.abs(v)).all()


@pytest.mark.parametrize("top", [65504.0, 2.0 ** 100, 448 * 2.0 ** 118, 3e38])
def test_numbers_of_huge_blocks(top):
    for dt in ("f16", "bf16", "f32") if top < 1e5 else ("bf16", "f32"):
        rng = gen(top, dt, "huge")
        x = rng.uniform(-1, 1, (40, 300)) * top
        x[:, [0, 130, 290]] = top
        x = cuda(x, DT[dt])
        for (q, s), rows in ((pw.pw_quant_f8(x), 1), (pw.pw_quant_f8_blocks(x), 128)):
            v, ref = f8.quotients(f64(x), rows)
            assert np.isfinite(f64(x)).all() and (np.abs(f64(s) - ref) <= ref * U).all()
            want = f8.e4m3(v)
            if dt != "f32":
                assert np.array_equal(f64(q), want)
            else:
                assert (np.abs(f64(q) - v) <= np.abs(want - v) + 2 * U * np.abs(v)).all()


def test_blocks_whose_scale_is_below_fp32():
    """448 x 2^-150 is the border: its scale is halfway between 0 and 2^-149, and goes to 0."""
    for n, scale in ((1, 0), (100, 0), (224, 0), (225, 1), (300, 1), (672, 2), (671, 1)):
        x = cuda(np.array([[n, -n, n // 2, 0]]) * V, torch.float32)
        for q, s in (pw.pw_quant_f8(x), pw.pw_quant_f8_blocks(x)):
            assert (f64(s) == scale * V).all()
            v, _ = f8.quotients(f64(x))
            assert np.array_equal(f64(q), f8.e4m3(v) if scale else 0 * v)
    x = torch.full((1, 130), INF, device="cuda")
    x[0, 128:] = V
    q, s = pw.pw_quant_f8(x)
    assert f64(s)[0, 0] == INF and f64(s)[0, 1] == 0 and (f64(q) == 0).all()
