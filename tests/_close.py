"""Comparison with a reference in 64 bits that nothing but a number can pass."""
import numpy as np

ROUND = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def assert_values(got, ref, dt, rel, extra=0.0):
    """got, rounded once to dt, within rel |ref| + extra of the finite ref; a NaN or an
    infinity in got fails."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    tol = np.abs(ref) * (rel + ROUND[dt]) + extra + (2.0 ** -25 if dt == "f16" else 1e-38)
    assert np.isfinite(ref).all() and got.shape == ref.shape
    ok = np.abs(got - ref) <= tol
    assert ok.all(), (int((~ok).sum()), float(np.abs(got - ref).max()))
