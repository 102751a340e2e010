"""pw_rms_norm on rows at the ends of the number range, against the fp64 oracle.

The tolerances are those of test_gpu_operators.py: a sum of squares off by 64 + 10
roundings of 2^-24, halved by the root, and five more operations."""
import itertools

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
def test_rows_of_zeros_without_eps(T, H):
    for dt, res in itertools.product(["f16", "bf16", "f32"], [False, True]):
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


def _row(kind, rng, H):
    n = rng.normal(0, 1, H)
    return {"large": n * 1e20, "largest": np.clip(n, -3, 3) * 1e38, "sum": n * 1e15, "small": n * 1e-25, "smaller": n * 1e-35,
            "one_large": np.where(np.arange(H) == H // 2, 1e25, n), "one_normal": np.where(np.arange(H) == H // 3, 1.0, n * 1e-25),
            "normal": n, "one_small": np.where(np.arange(H) == H - 1, 1e-30, 0.0)}[kind]


KINDS = ["large", "largest", "sum", "small", "smaller", "one_large", "one_normal", "normal", "one_small"]


@pytest.mark.parametrize("T,H", SHAPES)
def test_rows_whose_squares_leave_the_range(T, H):
    for dt, eps, res in itertools.product(["bf16", "f32"], [0.0, 1e-6], [False, True]):
        rng = np.random.default_rng([T, H])
        a = np.stack([_row(KINDS[t % len(KINDS)], rng, H) for t in range(max(T, len(KINDS)))])
        x = torch.as_tensor(a).to(DT[dt]).cuda()
        r = torch.as_tensor(a[:, ::-1] * 0.5).to(DT[dt]).cuda() if res else None
        w = torch.as_tensor(rng.normal(1, 0.1, H)).to(DT[dt]).cuda()
        # the sum as the kernel has it: fp32, one rounding
        s = (x.float() + (r.float() if res else 0.0)).double().cpu().numpy()
        out = torch.empty_like(x)
        got = pw.pw_rms_norm_i8(x, w, eps, residual=r, out=out)
        rel = 64 * U
        if res:
            assert torch.equal(got[2], torch.as_tensor(s).to(torch.float32).to(DT[dt]).cuda())
            # the residual stream updated in place
            out2, s2 = pw.pw_rms_norm(x, w, eps, residual=r, sum_out=r)
            assert torch.equal(out2.view(torch.uint8), out.view(torch.uint8)) and torch.equal(s2, got[2])
        # a sum that fp32 does not hold is an infinity, and has no scale
        inf = np.isinf(s)
        none, keep = inf.any(1), ~inf.any(1)
        q, sc = f64(got[0]), f64(got[1])
        assert np.isnan(f64(out)[inf]).all() and (f64(out)[none][~inf[none]] == 0).all()
        assert np.isnan(sc[none]).all() and (q[none] == 0).all()
        out, q, sc, (_, y) = f64(out)[keep], q[keep], sc[keep], ops.rms_norm(s[keep], f64(w), eps)
        # elements 2^-100 and more below the largest may be lost
        tiny = np.abs(y).max(1, keepdims=True) * 2.0 ** -100 + 1e-38
        assert (np.abs(out - y) <= np.abs(y) * (rel + ROUND[dt]) + tiny).all()
        steps, scale = ops.quant_i8(y)
        assert (np.abs(sc - scale) <= scale * (rel + 2 * U) + 1e-43).all()
        assert (np.abs(q - steps) <= 0.5 + 127 * (rel + 4 * U)).all()


@pytest.mark.parametrize("T,H", SHAPES)
def test_a_weight_that_is_no_number_spoils_its_own_element_only(T, H):
    for dt, bad in itertools.product(["f16", "bf16", "f32"], [float("inf"), float("nan")]):
        rng = np.random.default_rng([T, H, 3])
        x = torch.as_tensor(rng.normal(0, 2, (T, H))).to(DT[dt]).cuda()
        w = torch.as_tensor(rng.normal(1, 0.1, H)).to(DT[dt]).cuda()
        at = H // 2
        w[at] = bad
        y = f64(pw.pw_rms_norm(x, w, 1e-6))
        q, s = pw.pw_rms_norm_i8(x, w, 1e-6)
        assert not np.isfinite(y[:, at]).any() and not torch.isfinite(s).any() and (q == 0).all()
        w[at] = 0
        ref = ops.rms_norm(f64(x), f64(w), 1e-6)[1]
        keep = np.arange(H) != at
        assert (np.abs(y - ref)[:, keep] <= (np.abs(ref) * (64 * U + ROUND[dt]) + 2.0 ** -25)[:, keep]).all()


@pytest.mark.parametrize("T,H", SHAPES)
def test_rows_with_infinities_and_nan(T, H):
    """As the formula gives: 0 beside an infinity (a finite number by an infinite root),
    NaN at it; a NaN is everywhere.  No scale, and q 0."""
    for dt in ("f16", "bf16", "f32"):
        rng = np.random.default_rng([T, H, 5])
        x = torch.as_tensor(rng.normal(0, 2, (T, H))).to(DT[dt]).cuda()
        w = torch.as_tensor(rng.normal(1, 0.1, H)).to(DT[dt]).cuda()
        x[0, H // 2], x[1, 0], x[2, H - 1] = float("inf"), float("nan"), -float("inf")
        y = pw.pw_rms_norm(x, w, 1e-6)
        q, s = pw.pw_rms_norm_i8(x, w, 1e-6)
        for t, at in ((0, H // 2), (2, H - 1)):
            assert torch.isnan(y[t, at]) and (y[t, :at] == 0).all() and (y[t, at + 1:] == 0).all()
        assert torch.isnan(y[1]).all() and torch.isnan(s[:3]).all() and (q[:3] == 0).all()
        assert torch.isfinite(y[3:]).all() and torch.isfinite(s[3:]).all()