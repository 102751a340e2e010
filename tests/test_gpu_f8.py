"""The operators of an expert layer in 8-bit floating point against the fp64 oracle.

Tolerances.  U = 2^-24 is fp32's rounding; outputs are rounded once to their type
(relative 2^-11, 2^-8, U; 2^-25 absolute for fp16's subnormals).  Before that:
 * product: terms are exact in fp32.  A block adds 128 of them, each addition off by at
   most 2 U (a tensor core may cut instead of rounding), then two factors and the sum
   over blocks: (256 + blocks + 4) U of the sum of the absolute products; split sums of
   up to 8 parts add 8 U;
 * quantiser: scales by U; 16-bit inputs give the e4m3 number nearest to the exact
   quotient, 32-bit ones too but where it lies within 2 U of halfway; silu(gate) * up is
   off by e = (8 + |g| (1 - sigmoid(g))) U: 2 U each for exponential and reciprocal, U for
   the sum and each product, and the rounding of the exponential's argument g log2 e, by
   |g log2 e| U, changes 2^argument by |g| U and the sigmoid by 1 - sigmoid of that.  The
   block's largest is off as much: half a step and (2 e + 4 U) 448;
 * routing: an exponential is off by 2 U and its argument by |x - max| U, at most 32 U
   here; sums of E terms by E U;
 * weighted sum: (k + 2) U of the sum of the absolute terms.
"""
import numpy as np
import pytest
import torch

import any_precision_weight_gb300 as pw
from any_precision_weight_gb300.guard import GuardSet
from oracle import f8

from test_gpu_operators import DT, ROUND, U, Framed, f64, gen

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
INF, NAN = float("inf"), float("nan")


def cuda(a, dtype):
    return torch.as_tensor(np.ascontiguousarray(a)).to(dtype).cuda()


def near(got, ref, dt, tol):
    tol = tol + np.abs(ref) * ROUND[dt] + (2.0 ** -25 if dt == "f16" else 1e-38)
    got = f64(got)
    assert np.isfinite(ref).all() and np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) - tol).max())


def values(rng, *shape):
    """e4m3 numbers of all sizes on the GPU, rows on 16-byte boundaries."""
    q = pw.rows_f8(*shape)
    q.copy_(cuda(rng.normal(0, 1, shape) * 2.0 ** rng.integers(-8, 8, shape), torch.float32).clamp(-448, 448).to(F8))
    return q


def scales(rng, *shape):
    return cuda(rng.uniform(0.5, 2.0, shape) * 2.0 ** rng.integers(-6, 3, shape), torch.float32)


def product_tol(size, K, dt):
    return size * (256 + f8.blocks(K) + 12) * U


# ---------------------------------------------------------------- quantisers

ROWS = [(1, 1), (1, 128), (3, 129), (5, 1411), (17, 2048), (2, 14336), (33, 100), (300, 72)]


def check_q(q, s, x, dt, rows=1):
    v, ref = f8.quotients(x, rows)
    assert (np.abs(f64(s) - ref) <= ref * U).all()
    want, got = f8.e4m3(v), f64(q)
    if dt != "f32":
        assert np.array_equal(got, want)
    else:
        assert (np.abs(got - v) <= np.abs(want - v) + 2 * U * 448).all()


@pytest.mark.parametrize("T,K", ROWS)
def test_rows(T, K):
    for dt in DT:
        rng = gen(T, K, dt)
        x = cuda(rng.normal(0, 1, (T, K)) * 2.0 ** rng.integers(-3, 4, (T, K)), DT[dt])
        q, s = pw.pw_quant_f8(x)
        check_q(q, s, f64(x), dt)
        rows = cuda(rng.integers(0, 3 * T, 2 * T + 1), torch.int32)
        q, s = pw.pw_quant_f8(x, rows=rows, per=3)
        check_q(q, s, f64(x)[rows.cpu().numpy() // 3], dt)
        # a padded matrix that starts anywhere, into framed outputs
        wide = torch.zeros(T, K + 5, dtype=DT[dt], device="cuda")
        wide[:, 3:3 + K] = x
        fq, fs = Framed(T, K, torch.uint8, pad=3, off=1), Framed(T, f8.blocks(K), torch.float32, pad=1)
        pw.pw_quant_f8(wide[:, 3:3 + K], q=fq.view.view(F8), scale=fs.view)
        check_q(fq.view.view(F8), fs.view, f64(x), dt)
        assert fq.intact() and fs.intact()


def check_silu(q, s, x):
    g = f64(x)[:, :x.shape[1] // 2]
    with np.errstate(over="ignore"):   # e^|g| may be infinite, and what is divided by it 0
        e = (8 + np.abs(g) / (1 + np.exp(g))).max() * U   # 1 - sigmoid(g) = 1 / (1 + e^g)
        v, ref = f8.quotients(f8.silu_up(f64(x)))
    assert (np.abs(f64(s) - ref) <= ref * (e + 2 * U)).all()
    assert (np.abs(f64(q) - v) <= np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) + (2 * e + 4 * U) * 448).all()


@pytest.mark.parametrize("T,K", ROWS)
def test_silu_rows(T, K):
    for dt in DT:
        x = cuda(gen(T, K, dt, "silu").normal(0, 2, (T, 2 * K)), DT[dt])
        q, s = pw.pw_silu_quant_f8(x)
        check_silu(q, s, x)


@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (129, 257), (300, 1411), (1000, 64), (64, 3000)])
def test_blocks(N, K):
    for dt in DT:
        w = cuda(gen(N, K, dt, "w").normal(0, 0.02, (N, K)), DT[dt])
        fq, fs = Framed(N, K, torch.uint8, pad=(-K) % 16 + 16), Framed(f8.blocks(N), f8.blocks(K), torch.float32, pad=2)
        pw.pw_quant_f8_blocks(w, q=fq.view.view(F8), scale=fs.view)
        check_q(fq.view.view(F8), fs.view, f64(w), dt, 128)
        assert fq.intact() and fs.intact()


def test_silu_of_far_gates():
    """Gates of any size: no overflow, and a gate of -inf or NaN has that scale."""
    for dt in DT:
        top = {"f16": 6e4, "bf16": 1e38, "f32": 1e38}[dt]
        g = np.array([top, 100.0, 20.0, 0.0, -0.0, -20.0, -88.0, -88.7, -100.0, -top])
        x = cuda(np.concatenate([g, np.full(10, 1e-3)])[None], DT[dt])
        q, s = pw.pw_silu_quant_f8(x)
        check_silu(q, s, x)
        x[0, 2] = -INF
        q, s = pw.pw_silu_quant_f8(x)
        assert np.isnan(f64(s)).all() and (f64(q) == 0).all()


def test_rows_of_nothing_and_of_no_numbers():
    for dt in DT:
        x = torch.ones(6, 300, dtype=DT[dt], device="cuda")
        x[0] = 0
        x[1, 130] = INF
        x[2, 299] = -INF
        x[3, 0] = NAN
        x[4, :128] = -0.0
        q, s = pw.pw_quant_f8(x)
        q, s = f64(q), f64(s)
        one = np.float64(np.float32(1 / 448))
        assert (q[0] == 0).all() and (s[0] == 0).all()
        assert (q[1, 128:256] == 0).all() and s[1, 1] == INF and s[1, 0] == one and (q[1, :128] == 448).all()
        assert (q[2, 256:] == 0).all() and s[2, 2] == INF
        assert (q[3, :128] == 0).all() and np.isnan(s[3, 0]) and s[3, 1] == one
        assert (q[4, :128] == 0).all() and s[4, 0] == 0 and (q[5] == 448).all()
        bq, bs = pw.pw_quant_f8_blocks(x)
        assert np.isnan(f64(bs)[0, 0]) and f64(bs)[0, 1] == INF and (f64(bq) == 0).all()


def test_rows_at_the_ends_of_the_range():
    for dt, top in (("f16", 65504.0), ("bf16", 2.0 ** 127), ("f32", 3e38), ("f16", 2.0 ** -24), ("bf16", 2.0 ** -126),
                    ("f32", 2.0 ** -126), ("bf16", 2.0 ** -100)):
        x = cuda(np.array([[1.0, -0.5, 0.25, 0.0, 0.75] * 30]) * top, DT[dt])
        q, s = pw.pw_quant_f8(x)
        check_q(q, s, f64(x), dt) if top > 1e-30 else None
        # the scale may lie among fp32's subnormals: what it stands for is then off by half a step of those
        assert (np.abs(f64(q) * f64(s).repeat(128, 1)[:, :150] - f64(x)) <= np.abs(f64(x)) * 2.0 ** -4 + 448 * 2.0 ** -150).all()


def test_sources_out_of_range_are_rows_of_zeros():
    x = torch.ones(4, 200, dtype=torch.float16, device="cuda")
    rows = cuda(np.array([0, 7, 8, -1, 2**31 - 1, -2**31]), torch.int32)
    q, s = pw.pw_quant_f8(x, rows=rows, per=2)
    assert (f64(q)[:2] == 448).all() and (f64(q)[2:] == 0).all() and (f64(s)[2:] == 0).all()


# ---------------------------------------------------------------- products

PRODUCTS = [(1, 1, 1), (1, 16, 128), (2, 17, 127), (7, 60, 2048), (8, 1000, 1411), (9, 129, 300), (16, 2048, 1408),
            (17, 300, 4096), (31, 33, 5000), (33, 60, 4096), (48, 700, 129), (64, 1281, 1040), (65, 4100, 2049),
            (100, 257, 256), (128, 2000, 200), (129, 300, 20000), (201, 2891, 1411), (300, 1030, 3000), (513, 640, 64),
            (700, 90, 16), (1025, 1003, 411)]


@pytest.mark.parametrize("T,N,K", PRODUCTS)
def test_linear(T, N, K):
    for dt in DT:
        rng = gen(T, N, K, dt, "linear")
        x, w = values(rng, T, K), values(rng, N, K)
        xs, ws = scales(rng, T, f8.blocks(K)), scales(rng, f8.blocks(N), f8.blocks(K))
        b = cuda(rng.normal(0, 1, N), DT[dt]) if T % 2 else None
        # the size where fp16 holds every sum
        if dt == "f16":
            xs *= 2.0 ** -14
        out = Framed(T, N, DT[dt], pad=T % 3, off=T % 2)
        pw.pw_linear_f8(x, xs, w, ws, bias=b, out=out.view)
        ref, size = f8.linear(f64(x), f64(xs), f64(w), f64(ws), None if b is None else f64(b))
        near(out.view, ref, dt, product_tol(size, K, dt) + 2 * U * np.abs(ref))
        assert out.intact()


GROUPS = [([1], 16, 128), ([0, 3, 0, 1], 130, 200), ([0] * 7 + [5], 60, 1411), ([2, 0, 9, 17, 1, 0, 33], 300, 257),
          ([64, 1, 130, 0, 257], 513, 384), ([0, 0, 700], 90, 1000), ([5] * 60, 64, 130), ([1] * 512, 40, 64),
          ([300, 20], 2048, 1408), ([0], 8, 8), ([0, 0, 0], 300, 300)]


@pytest.mark.parametrize("counts,N,K", GROUPS)
def test_grouped(counts, N, K):
    E, R = len(counts), sum(counts)
    for dt in DT:
        rng = gen(E, R, N, K, dt, "grouped")
        first, rest = int(rng.integers(0, 3)), int(rng.integers(1, 4))   # rows before and behind every group
        T = first + R + rest
        x, w = values(rng, T, K), values(rng, E, N, K)
        xs, ws = scales(rng, T, f8.blocks(K)), scales(rng, E, f8.blocks(N), f8.blocks(K))
        # NaN in rows that belong to no group
        for a, z in ((0, first), (first + R, T)):
            x.view(torch.uint8)[a:z] = 0x7F
            xs[a:z] = NAN
        if dt == "f16":
            xs *= 2.0 ** -14
        b = cuda(rng.normal(0, 1, (E, N)), DT[dt]) if E % 2 else None
        off = first + np.concatenate([[0], np.cumsum(counts)])
        out = Framed(T, N, DT[dt], pad=1)
        pw.pw_grouped_linear_f8(x, xs, w, ws, cuda(off, torch.int32), bias=b, out=out.view)
        assert out.intact()
        assert (f64(out.view)[:first] == 77).all() and (f64(out.view)[first + R:] == 77).all()
        for e in range(E):
            a, z = off[e], off[e + 1]
            if z > a:
                ref, size = f8.linear(f64(x)[a:z], f64(xs)[a:z], f64(w[e]), f64(ws[e]), None if b is None else f64(b)[e])
                near(out.view[a:z], ref, dt, product_tol(size, K, dt) + 2 * U * np.abs(ref))


# sizes that pairs of CTAs take in tiles of 256 x 256, the last of a group's rows few
LAST = [([257], 9728, 256), ([300], 9500, 300), ([320], 9728, 130), ([321], 9600, 128), ([384], 9665, 200), ([385], 9728, 200),
        ([513], 9700, 270), ([1100], 9728, 130), ([1, 256, 0, 130, 385, 33, 64, 131], 2048, 300),
        ([65, 128, 129, 127, 300, 2, 63, 186], 4003, 257)]


@pytest.mark.parametrize("counts,N,K", LAST)
def test_last_rows(counts, N, K):
    E, T = len(counts), sum(counts)
    for dt in DT:
        rng = gen(E, T, N, K, dt, "last")
        x, w = values(rng, T, K), values(rng, E, N, K)
        xs, ws = scales(rng, T, f8.blocks(K)), scales(rng, E, f8.blocks(N), f8.blocks(K))
        if dt == "f16":
            xs *= 2.0 ** -14
        b = cuda(rng.normal(0, 1, (E, N)), DT[dt])
        off = np.concatenate([[0], np.cumsum(counts)])
        for pad in (0, 1):   # stores by TMA, and channel by channel
            out = Framed(T, N, DT[dt], pad=pad + (-N) % 8)
            if E == 1:
                pw.pw_linear_f8(x, xs, w[0], ws[0], bias=b[0], out=out.view)
            else:
                pw.pw_grouped_linear_f8(x, xs, w, ws, cuda(off, torch.int32), bias=b, out=out.view)
            assert out.intact()
            if pad == 0:
                want = out.view.clone()
            assert torch.equal(out.view, want)
        for e in range(E):
            a, z = off[e], off[e + 1]
            if z > a:
                ref, size = f8.linear(f64(x)[a:z], f64(xs)[a:z], f64(w[e]), f64(ws[e]), f64(b)[e])
                near(want[a:z], ref, dt, product_tol(size, K, dt) + 2 * U * np.abs(ref))


@pytest.mark.parametrize("T,N", [(4, 64), (40, 300), (400, 2000), (3000, 2000)])
def test_offsets_out_of_order(T, N):
    """Cut to [0, T]; nothing beside the rows is touched."""
    g = GuardSet(4096)
    rng = gen(T, "offsets")
    E, K = 4, 128 if T < 3000 else 640
    x, w, xs, ws = values(rng, T, K), values(rng, E, N, K), scales(rng, T, K // 128), scales(rng, E, f8.blocks(N), K // 128)
    out = g.alloc(T * N * 4, "cuda", "out").view(torch.float32).view(T, N)
    again = torch.empty_like(out)
    for off in ([-5, 2, 1, T + 9, 2 ** 31 - 1], [T + 1, 0, -2 ** 31, 3, 2], [7, 7, 7, 7, 7], [2 ** 31 - 1] * 5, [0, T, 0, T, 0],
                [0] * 5, [3, 1, T // 2, 0, T - 1]):
        out.fill_(77)
        pw.pw_grouped_linear_f8(x, xs, w, ws, cuda(np.array(off), torch.int32), out=out)
        assert g.corrupted() == []
        order = np.clip(off, 0, T)
        if (np.diff(order) < 0).any():
            continue
        again.fill_(77)
        pw.pw_grouped_linear_f8(x, xs, w, ws, cuda(order, torch.int32), out=again)
        assert torch.equal(out, again)
        left = torch.cat([again[:order[0]], again[order[-1]:]])
        assert (left == 77).all()


def test_rows_with_no_numbers_stay_alone():
    """A NaN or an infinity in one row's scale, or behind K, reaches no other row."""
    for T in (3, 40, 300):
        rng = gen(T, "nan")
        K = 200
        x, w = values(rng, T, K), values(rng, 300, K)
        xs, ws = scales(rng, T, 2), scales(rng, 3, 2)
        want = pw.pw_linear_f8(x, xs, w, ws, out_dtype=torch.float32)
        for q in (x, w):
            torch.as_strided(q.view(torch.uint8), (q.shape[0], 8), (208, 1), 200).fill_(0x7F)   # behind K
        xs[1, 1], xs[T - 1, 0] = NAN, INF
        got = pw.pw_linear_f8(x, xs, w, ws, out_dtype=torch.float32)
        assert torch.isnan(got[1]).all() and not torch.isfinite(got[T - 1]).any()
        keep = [t for t in range(T) if t not in (1, T - 1)]
        assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("K", [1, 15, 17, 129, 201, 206, 255, 1411])
def test_bytes_behind_rows(K):
    """NaN in them change nothing: few rows, single CTAs and pairs, rows in groups."""
    for T, N in ((3, 300), (16, 70), (40, 3000), (129, 9728), (300, 9728)):
        rng = gen(T, K, "behind")
        x, w = values(rng, T, K), values(rng, N, K)
        xs, ws = scales(rng, T, f8.blocks(K)), scales(rng, f8.blocks(N), f8.blocks(K))
        off = cuda(np.array([0, T // 3, T]), torch.int32)
        g = lambda: pw.pw_grouped_linear_f8(x, xs, w[None].expand(2, N, K), ws[None].expand(2, -1, -1), off,
                                            out_dtype=torch.float32)
        outs = []
        for byte in (0, 0x7F):
            for q in (x, w):
                ld = q.stride(0)
                torch.as_strided(q.view(torch.uint8), (q.shape[0], ld - K), (ld, 1), K).fill_(byte)
            outs.append((pw.pw_linear_f8(x, xs, w, ws, out_dtype=torch.float32), g()))
        for a, b in zip(*outs):
            assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("T,K", [(1, 1), (5, 129), (33, 100), (300, 1408), (7, 14336)])
def test_silu_and_gathered_rows_in_frames(T, K):
    for dt in DT:
        rng = gen(T, K, dt, "frames")
        x = torch.zeros(T + 2, 2 * K + 3, dtype=DT[dt], device="cuda")[1:T + 1, 1:1 + 2 * K]
        x.copy_(cuda(rng.normal(0, 2, (T, 2 * K)), DT[dt]))
        for pad, off in ((0, 0), ((-K) % 16 + 16, 0), (5, 1)):
            fq, fs = Framed(T, K, torch.uint8, pad=pad, off=off), Framed(T, f8.blocks(K), torch.float32, pad=pad)
            pw.pw_silu_quant_f8(x, q=fq.view.view(F8), scale=fs.view)
            check_silu(fq.view.view(F8), fs.view, x)
            assert fq.intact() and fs.intact()
            rows = cuda(rng.integers(0, 2 * T, T), torch.int32)
            fq, fs = Framed(T, K, torch.uint8, pad=pad, off=off), Framed(T, f8.blocks(K), torch.float32, pad=pad)
            pw.pw_quant_f8(x[:, :K], rows=rows, per=2, q=fq.view.view(F8), scale=fs.view)
            check_q(fq.view.view(F8), fs.view, f64(x)[rows.cpu().numpy() // 2, :K], dt)
            assert fq.intact() and fs.intact()


def test_one_group_is_the_plain_product():
    for T in (5, 70, 500):
        rng = gen(T, "one")
        x, w, xs, ws = values(rng, T, 640), values(rng, 500, 640), scales(rng, T, 5), scales(rng, 4, 5)
        a = pw.pw_linear_f8(x, xs, w, ws, out_dtype=torch.float32)
        b = pw.pw_grouped_linear_f8(x, xs, w[None], ws[None], cuda(np.array([0, T]), torch.int32), out_dtype=torch.float32)
        ref, size = f8.linear(f64(x), f64(xs), f64(w), f64(ws))
        for o in (a, b):
            near(o, ref, "f32", product_tol(size, 640, "f32"))


@pytest.mark.parametrize("T,N,K", [(4000, 3, 60001), (4100, 11000, 16), (17, 60, 700000)])
def test_thin_products(T, N, K):
    rng = gen(T, N, K, "thin")
    x, w = values(rng, T, K), values(rng, N, K)
    xs, ws = scales(rng, T, f8.blocks(K)), scales(rng, f8.blocks(N), f8.blocks(K))
    out = pw.pw_linear_f8(x, xs, w, ws, out_dtype=torch.float32)
    t = np.unique(np.linspace(0, T - 1, 200).astype(int))
    ref, size = f8.linear(f64(x[t]), f64(xs[t]), f64(w), f64(ws))
    near(out[t], ref, "f32", product_tol(size, K, "f32"))


# ---------------------------------------------------------------- routing and the weighted sum

def check_route(r, x, k, renorm):
    ref = f8.route(x, k, renorm)
    for name in ("idx", "offsets", "perm", "inv"):
        assert np.array_equal(f64(getattr(r, name)), ref[name]), name
    assert (np.abs(f64(r.weight) - ref["weight"]) <= ref["weight"] * (2 * 34 + x.shape[1] + 4) * U + 1e-38).all()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (4, 60, 4), (3, 33, 33), (128, 8, 8), (129, 8, 8), (300, 60, 4),
                                   (17, 65, 64), (500, 129, 5), (70, 256, 8), (33, 257, 40), (9, 512, 512), (3000, 100, 3)])
@pytest.mark.parametrize("renorm", [False, True])
def test_route(T, E, k, renorm):
    rng = gen(T, E, k)
    # coarse logits: ties in every row
    x = np.round(rng.normal(0, 3, (T, E)).clip(-16, 16) * 4) / 4
    wide = torch.full((T, E + 3), NAN, device="cuda")
    wide[:, 1:1 + E] = cuda(x, torch.float32)
    check_route(pw.pw_route(wide[:, 1:1 + E], k, renorm), x, k, renorm)
    same = np.zeros((T, E))
    same[:, ::2] = -0.0   # both zeros are equal
    check_route(pw.pw_route(cuda(same, torch.float32), k, renorm), same, k, renorm)


def test_route_of_masked_rows():
    for T in (5, 400):
        x = gen(T, "mask").normal(0, 1, (T, 40))
        x[0] = -INF
        x[1, 3:] = -INF
        x[2, 5] = NAN
        x[3, [4, 9]] = INF
        x[4] = NAN
        x[T - 1, 0] = np.finfo(np.float32).min
        for renorm in (False, True):
            r = pw.pw_route(cuda(x, torch.float32), 6, renorm)
            check_route(r, x.astype(np.float32), 6, renorm)
            none = [0, 4] if T > 5 else [0]   # of 5 rows the last one has a number
            assert (f64(r.weight)[none] == 0).all() and (f64(r.weight)[1, 3:] == 0).all()


def test_route_as_the_layer_routes():
    """The same experts and order as the fused layer's own routing."""
    import synth
    from _layers import LIVE
    from any_precision_weight_gb300.model import load_expert_layer
    cfg = synth.CONFIGS["tiny"]
    m = pw.PagedMoE(1, cfg.E, cfg.H, cfg.I, guard=256)
    LIVE.append(m)
    load_expert_layer(m, 0, lambda e, kind: (synth.parent_indices(cfg, 0, e, kind), synth.parent_lut(cfg, 0, e, kind)),
                      synth.block_bits(cfg))
    for T in (1, 16, 200):
        x = torch.from_numpy(synth.tokens(cfg, T=T)).cuda()
        logits = cuda(gen(T, "layer").normal(0, 1, (T, cfg.E)), torch.float32)
        _, idx, weight, offsets, perm = m.pw_moe_forward(0, x, logits, cfg.top_k, cfg.renorm, routing=True)
        r = pw.pw_route(logits, cfg.top_k, cfg.renorm)
        for a, b in ((r.idx, idx), (r.offsets, offsets), (r.perm, perm)):
            assert torch.equal(a, b)
        assert (weight - r.weight).abs().max() <= 64 * U


@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 2, 4096), (4, 4, 2048), (7, 3, 1411), (300, 2, 264), (3, 8, 14336)])
def test_combine(T, k, H):
    for dy in DT:
        for do in DT:
            rng = gen(T, k, H, dy, do)
            y = cuda(rng.normal(0, 1, (T * k + 2, H)), DT[dy])
            w = cuda(rng.uniform(0, 1, (T, k)), torch.float32)
            inv = rng.permutation(T * k + 2)[:T * k]
            res = cuda(rng.normal(0, 1, (T, H)), DT[do]) if T != 7 else None
            out = Framed(T, H, DT[do], pad=T % 3)
            pw.pw_combine(y, w, cuda(inv, torch.int32), residual=res, out=out.view)
            ref, size = f8.combine(f64(y), f64(w), inv, None if res is None else f64(res))
            near(out.view, ref, do, size * (k + 2) * U)
            assert out.intact()
            if res is not None:   # in place
                assert torch.equal(pw.pw_combine(y, w, cuda(inv, torch.int32), residual=res, out=res), out.view)


def test_combine_leaves_out_what_has_no_weight_or_place():
    y = torch.full((3, 200), NAN, dtype=torch.float16, device="cuda")
    y[1] = 2
    w = cuda(np.array([[0.5, 0.0, 1.0, 1.0], [0.0] * 4]), torch.float32)
    inv = cuda(np.array([[1, 0, -1, 3], [0, 2, 2 ** 31 - 1, -2 ** 31]]), torch.int32)
    out = f64(pw.pw_combine(y, w, inv))
    assert (out[0] == 1).all() and (out[1] == 0).all()


# ---------------------------------------------------------------- together

def _layer(E, H, I, dt, seed):
    from any_precision_weight_gb300.model import F8Experts
    rng = gen(E, H, I, seed)
    up = cuda(rng.normal(0, H ** -0.5, (E, 2 * I, H)), DT[dt])
    down = cuda(rng.normal(0, I ** -0.5, (E, H, I)), DT[dt])
    return F8Experts(up, down), rng


def _check_layer(m, x, logits, k, renorm, residual, dt):
    """The layer against the oracle, stage by stage on what each stage read."""
    out, t = m.forward(x, logits, k, renorm, residual=residual, trace=True)
    T, E = logits.shape
    check_route(t.routing, f64(logits), k, renorm)
    off = t.routing.offsets.tolist()
    check_q(t.q, t.scale, f64(x)[f64(t.routing.perm).astype(int) // k], dt)
    check_silu(t.act, t.act_scale, t.up)
    for q, sc, w, ws, o in ((t.q, t.scale, m.gate_up, m.gate_up_scale, t.up), (t.act, t.act_scale, m.down, m.down_scale, t.y)):
        for e in range(E):
            a, z = off[e], off[e + 1]
            if z > a:
                ref, size = f8.linear(f64(q[a:z]), f64(sc[a:z]), f64(w[e]), f64(ws[e]))
                near(o[a:z], ref, dt, product_tol(size, q.shape[1], dt) + 2 * U * np.abs(ref))
    ref, size = f8.combine(f64(t.y), f64(t.routing.weight), t.routing.inv.cpu().numpy(), None if residual is None else f64(residual))
    near(out, ref, dt, size * (k + 2) * U)
    return out


@pytest.mark.parametrize("T,E,k,H,I,dt", [(1, 8, 2, 256, 512, "f16"), (5, 60, 4, 200, 136, "bf16"), (64, 8, 2, 256, 512, "f16"),
                                          (300, 16, 4, 264, 500, "bf16"), (1000, 8, 2, 256, 384, "f16")])
def test_expert_layer(T, E, k, H, I, dt):
    m, rng = _layer(E, H, I, dt, T)
    x, logits = cuda(rng.normal(0, 1, (T, H)), DT[dt]), cuda(rng.normal(0, 1, (T, E)), torch.float32)
    res = cuda(rng.normal(0, 1, (T, H)), DT[dt]) if T % 2 else None
    _check_layer(m, x, logits, k, True, res, dt)


@pytest.mark.parametrize("T", [3, 50, 500])
def test_expert_layer_as_a_graph_and_on_another_stream(T):
    m, rng = _layer(8, 256, 512, "f16", T)
    x, logits = cuda(rng.normal(0, 1, (T, 256)), torch.float16), cuda(rng.normal(0, 1, (T, 8)), torch.float32)
    want = m.forward(x, logits, 2, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = m.forward(x, logits, 2, True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = m.forward(x, logits, 2, True)
    # other inputs in the same places
    x2, l2 = cuda(rng.normal(0, 1, (T, 256)), torch.float16), cuda(rng.normal(0, 3, (T, 8)), torch.float32)
    want2 = m.forward(x2, l2, 2, True)
    x.copy_(x2)
    logits.copy_(l2)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap, want2)


def test_no_tokens():
    m, _ = _layer(8, 256, 512, "f16", 0)
    x = torch.empty(0, 256, dtype=torch.float16, device="cuda")
    r = pw.pw_route(torch.empty(0, 8, device="cuda"), 2)
    assert (r.offsets == 0).all() and r.offsets.numel() == 9
    assert m.forward(x, torch.empty(0, 8, device="cuda"), 2, True).shape == (0, 256)


@pytest.mark.parametrize("T,N,K", [(1, 60, 2048), (9, 300, 1000), (40, 1030, 520), (300, 520, 1411)])
def test_nothing_beside_the_outputs(T, N, K):
    g = GuardSet(4096)
    new = lambda shape, dt: g.alloc(max(1, int(np.prod(shape)) * torch.empty(0, dtype=dt).element_size()), "cuda",
                                    str(shape)).fill_(0xFF).view(dt).view(shape)
    rng = gen(T, N, K, "guards")
    x = cuda(rng.normal(0, 1, (T, K)), torch.float16)
    kb = f8.blocks(K)
    q, s = new((T, (K + 15) // 16 * 16), F8), new((T, kb), torch.float32)
    pw.pw_quant_f8(x, q=q[:, :K], scale=s)
    w, ws = pw.pw_quant_f8_blocks(cuda(rng.normal(0, 1, (N, K)), torch.float16))
    out = new((T, N), torch.float32)
    pw.pw_linear_f8(q[:, :K], s, w, ws, out=out)
    assert torch.isfinite(out).all()
    grouped = new((T, N), torch.float32)
    pw.pw_grouped_linear_f8(q[:, :K], s, w[None], ws[None], cuda(np.array([0, T]), torch.int32), out=grouped)
    assert torch.isfinite(grouped).all()
    i32, f32 = torch.int32, torch.float32
    r = pw.Routing(new((T, 3), i32), new((T, 3), f32), new((41,), i32), new((3 * T,), i32), new((3 * T,), i32))
    pw.pw_route(cuda(rng.normal(0, 1, (T, 40)), f32), 3, out=r)
    a, sa = new((T, K // 2), F8), new((T, f8.blocks(K // 2)), f32)
    pw.pw_silu_quant_f8(x[:, :K // 2 * 2], q=a, scale=sa)
    c = new((T, N), torch.float16)
    pw.pw_combine(out.repeat(3, 1), r.weight, r.inv, out=c)
    assert g.corrupted() == []
    assert torch.isfinite(c.float()).all() and torch.isfinite(sa).all()
