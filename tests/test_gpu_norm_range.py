"""pw_rms_norm on rows at the ends of the number range, against the fp64 oracle.

The tolerances are those of test_gpu_operators.py: a sum of squares off by 64 + 10
roundings of 2^-24, halved by the root, and five more operations."""
import numpy as np
import pytest
import torch

import any_precision_weight_gb300 as pw
from oracle import operators as ops

from test_gpu_operators import DT, ROUND, U, f64

pytestmark = pytest.mark.gpu

# rows of one CTA by elements and by vectors, persistent ones, rows read twice
SHAPES = [(4, 33), (4, 512), (4, 1411), (3, 9000), (400, 512), (400, 513), (400, 4096), (4, 70001), (3, 70008)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("res", [False, True])
def test_rows_of_zeros_without_eps(T, H, dt, res):
    x = torch.ones(T, H, device="cuda", dtype=DT[dt])
    x[0], x[2] = 0, -0.0
    w = torch.full((H,), 1.5, device="cuda", dtype=DT[dt])
    r = torch.zeros_like(x) if res else None
    y = pw.pw_rms_norm(x, w, 0.0, residual=r)
    q, s = pw.pw_rms_norm_i8(x, w, 0.0, residual=r)[:2]
    y = y[0] if res else y
    for t in (0, 2):
        assert (y[t] == 0).all() and s[t] == 0 and (q[t] == 0).all()
    assert (y[1] == 1.5).all() and (q[1] == 127).all()
    assert abs(s[1].item() * 127 - 1.5) <= 1.5 * 4 * U
