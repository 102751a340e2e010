"""The experts' weighted sum on top of its own output: residual and out one matrix.

Tolerance: as in test_gpu_f8.py, (k + 2) U of the sum of the absolute terms and the output's rounding.
"""
import pytest
import torch

import any_precision_weight_gb300 as pw
from oracle import f8

from test_gpu_f8 import cuda, near
from test_gpu_operators import DT, U, f64, gen

pytestmark = pytest.mark.gpu


# a slot to four with the tokens one by one; two tokens at a time (many tokens of one or two
# slots); columns over several CTAs; rows that start anywhere
@pytest.mark.parametrize("T,k,H,pad", [(1, 2, 4096, 0), (5, 8, 14336, 0), (300, 5, 264, 0), (1500, 2, 264, 8), (2001, 1, 2064, 0),
                                       (1300, 2, 1411, 1)])
def test_combine_onto_its_residual(T, k, H, pad):
    for dy in DT:
        for do in DT:
            rng = gen(T, k, H, dy, do, "in place")
            y = cuda(rng.normal(0, 1, (T * k, H)), DT[dy])
            w = cuda(rng.uniform(0, 1, (T, k)), torch.float32)
            inv = rng.permutation(T * k)
            at = cuda(inv, torch.int32)
            m = torch.zeros(T, H + pad, dtype=DT[do], device="cuda")
            m[:, :H] = cuda(rng.normal(0, 1, (T, H)), DT[do])
            res = m[:, :H].clone()
            apart = pw.pw_combine(y, w, at, residual=res)
            got = pw.pw_combine(y, w, at, residual=m[:, :H], out=m[:, :H])
            assert torch.equal(got, apart) and (m[:, H:] == 0).all()
            ref, size = f8.combine(f64(y), f64(w), inv, f64(res))
            near(apart, ref, do, size * (k + 2) * U)
