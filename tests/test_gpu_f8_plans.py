"""Every way in which the products in 8 bits are worked out, against the fp64 oracle: which one
a size takes depends on the GPU's multiprocessors and clusters, so each is asked for here.

K has more blocks (of 128 columns) than the kernel has stages, accumulators and places for
scales, in each part too where K is split; T and N end inside tiles of every shape; outputs lie
where stores go by TMA, 16 bytes at a time, and element by element.  Tolerances as in test_gpu_f8.py.
"""
import functools

import numpy as np
import pytest
import torch

import any_precision_weight_gb300 as pw
from oracle import f8

from test_gpu_f8 import cuda, near, product_tol, scales, values
from test_gpu_operators import DT, U, Framed, f64, gen

pytestmark = pytest.mark.gpu

SINGLE = [(1, rows, channels) for rows in (16, 32, 64, 128) for channels in (64, 128, 192, 256)]
PAIRS = [(2, 128, channels) for channels in (64, 128, 192, 256)]


@functools.lru_cache(maxsize=2)
def case(T, N, K, counts=()):
    """Operands, offsets, and for each output row the oracle's value and size without a bias."""
    rng = gen(T, N, K, *counts, "plans")
    E = max(1, len(counts))
    x, w = values(rng, T, K), values(rng, E, N, K)
    xs, ws = scales(rng, T, f8.blocks(K)), scales(rng, E, f8.blocks(N), f8.blocks(K))
    off = np.concatenate([[0], np.cumsum(counts)]).astype(int) if counts else np.array([0, T])
    ref, size = np.zeros((T, N)), np.zeros((T, N))
    for e in range(E):
        a, z = off[e], off[e + 1]
        if z > a:
            ref[a:z], size[a:z] = f8.linear(f64(x[a:z]), f64(xs[a:z]), f64(w[e]), f64(ws[e]))
    return x, xs, w, ws, cuda(off, torch.int32) if counts else None, off, rng.normal(0, 1, (E, N)), ref, size


def check(way, T, N, K, counts=(), types=DT):
    x, xs, w, ws, offsets, off, b, ref, size = case(T, N, K, counts)
    for dt in types:
        small = 2.0 ** -14 if dt == "f16" else 1.0   # the size where fp16 holds every sum
        bias = cuda(b, DT[dt])
        full = ref * small + np.repeat(f64(bias), np.diff(off), axis=0)
        for pad, at in ((-N % 8, 0), (3, 1)):
            out = Framed(T, N, DT[dt], pad=pad, off=at)
            pw.pw_debug_linear_f8(way, x, xs * small, w, ws, offsets, bias=bias, out=out.view)
            near(out.view, full, dt, product_tol(size * small, K, dt) + 2 * U * np.abs(full))
            assert out.intact(), way
    assert pw.pw_linear_f8_status() == 0


@pytest.mark.parametrize("ctas,rows,channels", SINGLE)
def test_single_ctas(ctas, rows, channels):
    for parts in (1, 2, 4):
        check((ctas, rows, channels, parts), 141, 451, 6700)
    check((ctas, rows, channels, 1), 300, 700, 1931)


@pytest.mark.parametrize("ctas,rows,channels", PAIRS)
def test_pairs(ctas, rows, channels):
    for parts in (1, 2, 4):
        check((ctas, rows, channels, parts), 300, 451, 6700)   # the last pair's rows few
    for T in (450, 512, 129, 70):   # many; all; of two tiles the second has one; one CTA of the pair without rows
        for parts in (1, 2):
            check((ctas, rows, channels, parts), T, 700, 1931, types=["bf16"])


@pytest.mark.parametrize("ctas,rows,channels", SINGLE + PAIRS)
def test_rows_in_groups(ctas, rows, channels):
    check((ctas, rows, channels, 1), 757, 451, 1931, (5, 0, 130, 300, 64, 1, 257))


@pytest.mark.parametrize("parts", [1, 2, 4, 8])
def test_few_rows(parts):
    for rows in (8, 16):
        for share in (1, 2, 5):
            check((0, rows, share, parts), 37, 75, 3001)
            check((0, rows, share, parts), 63, 83, 1931, (0, 37, 1, 8, 17))


def test_many_more_tiles_than_ctas():
    """Rings and accumulators go on from one tile to the next, with an odd number of blocks."""
    for way in ((1, 128, 64, 1), (1, 32, 128, 1), (2, 128, 256, 1), (2, 128, 192, 1)):
        check(way, 1500, 2500, 1931, types=["bf16"])
        check(way, 1501, 1300, 400, (700, 1, 0, 300, 250, 250), types=["bf16"])
