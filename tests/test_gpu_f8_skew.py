"""Rows that all, or nearly all, go to one expert, at sizes whose way is chosen for a few rows to
each (two rows to an expert, or less, on average).  Tolerances as in test_gpu_f8.py."""
import numpy as np
import pytest
import torch

import any_precision_weight_gb300 as pw
from oracle import f8

from test_gpu_f8 import cuda, near, product_tol, scales, values
from test_gpu_operators import DT, U, Framed, f64, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,T,N,K", [(128, 256, 200, 1408), (512, 1024, 75, 300), (60, 61, 130, 2900), (8, 16, 1000, 4096)])
@pytest.mark.parametrize("hot", ["first", "last", "two"])
def test_rows_of_one_expert(E, T, N, K, hot):
    counts = np.zeros(E, int)
    if hot == "two":
        counts[[E // 2, E // 2 + 1]] = T - T // 3, T // 3
    else:
        counts[0 if hot == "first" else -1] = T
    off = np.concatenate([[0], np.cumsum(counts)])
    for dt in DT:
        rng = gen(E, T, N, K, hot, dt, "skew")
        x, w = values(rng, T, K), values(rng, E, N, K)
        xs, ws = scales(rng, T, f8.blocks(K)), scales(rng, E, f8.blocks(N), f8.blocks(K))
        if dt == "f16":
            xs *= 2.0 ** -14
        out = Framed(T, N, DT[dt], pad=1)
        pw.pw_grouped_linear_f8(x, xs, w, ws, cuda(off, torch.int32), out=out.view)
        assert out.intact()
        for e in np.flatnonzero(counts):
            a, z = off[e], off[e + 1]
            ref, size = f8.linear(f64(x)[a:z], f64(xs)[a:z], f64(w[e]), f64(ws[e]))
            near(out.view[a:z], ref, dt, product_tol(size, K, dt) + 2 * U * np.abs(ref))
