"""The operators around the layer against the fp64 oracle.

Tolerances.  U = 2^-24 is fp32's rounding.  Outputs are rounded once to their
type: relative 2^-11 (fp16), 2^-8 (bf16), U (fp32), and 2^-25 absolute for
fp16's subnormals.  Before that rounding:
 * norm: sum of H squares in fp32 over at most 64 terms a thread and 10 levels
   of a tree: (64 + 10) U relative, halved by the square root; five more
   operations: 64 U in all;
 * quantiser: the steps v * 127 / max are off by at most 4 U relative, so a
   step count of at most 127 by 127 * 64 U (norm's max included), and the
   rounding to whole numbers by 0.5;
 * product: the int32 sum is exact; its conversion and two factors: 3 U;
 * log probabilities: a sum of n = V / 256 + 32 terms a thread, each off by
   4 U (exp2 of an argument rounded relative to at most 16): (n + 24) U
   relative in s and u; logprob and entropy add their own roundings.
"""
import zlib

import numpy as np
import pytest
import torch

import any_precision_weight_gb300 as pw
from oracle import operators as ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": U}
INF = float("inf")


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def gen(*key):
    return np.random.default_rng([71, *[zlib.crc32(k.encode()) if isinstance(k, str) else int(k) for k in key]])


def place(a, dtype, pad=0, off=0):
    """The array as a CUDA matrix that starts `off` elements into rows of len + pad + off."""
    a = torch.as_tensor(np.ascontiguousarray(a))
    base = torch.zeros(a.shape[0], off + a.shape[1] + pad, dtype=dtype, device="cuda")
    v = base[:, off:off + a.shape[1]]
    v.copy_(a.to(dtype))
    return v


class Framed:
    """An output matrix inside a larger one whose other bytes must not change."""

    def __init__(self, T, H, dtype, pad=0, off=0):
        self.raw = torch.full((T + 2, H + pad + off), 77, dtype=dtype, device="cuda")
        self.view = self.raw[1:T + 1, off:off + H]

    def intact(self):
        r = self.raw.clone()
        T = r.shape[0] - 2
        H = self.view.shape[1]
        off = self.view.storage_offset() - r.shape[1]
        r[1:T + 1, off:off + H] = 77
        return bool((r == 77).all())


def check_out(got, ref, dt, rel, extra=0.0):
    tol = np.abs(ref) * (rel + ROUND[dt]) + extra + (2.0 ** -25 if dt == "f16" else 1e-38)
    bad = np.abs(f64(got) - ref) > tol
    assert not bad.any(), (int(bad.sum()), float(np.abs(f64(got) - ref).max()))


def check_q(q, scale, y, rel):
    steps, ref = ops.quant_i8(y)
    s = f64(scale)
    assert (np.abs(s - ref) <= ref * (rel + 2 * U)).all()
    err = np.abs(f64(q) - steps)
    assert err.max(initial=0) <= 0.5 + 127 * (rel + 4 * U)
    assert np.abs(f64(q)).max(initial=0) <= 127


NORMS = [(1, 1), (1, 128), (3, 31), (2, 256), (5, 1411), (4, 2048), (7, 4096), (2, 8200), (3, 14336), (2, 16384),
         (1, 40000), (300, 64), (2, 70001)]


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("res", [False, True])
def test_norm(T, H, dt, res):
    rng = gen(T, H, dt, res)
    x = place(rng.normal(0, 2, (T, H)), DT[dt])
    w = torch.as_tensor(rng.normal(1, 0.3, H)).to(DT[dt]).cuda()
    r = place(rng.normal(0, 3, (T, H)), DT[dt]) if res else None
    s, y = ops.rms_norm(f64(x), f64(w), 1e-5, f64(r) if res else None)
    rel = 64 * U
    got = pw.pw_rms_norm(x, w, 1e-5, residual=r)
    if res:
        check_out(got[1], s, dt, U)
        got = got[0]
    check_out(got, y, dt, rel, extra=np.abs(w.double().cpu().numpy()) * 4 * U if res else 0.0)
    i8 = pw.pw_rms_norm_i8(x, w, 1e-5, residual=r, out=torch.empty_like(x))
    check_q(i8[0], i8[1], y, rel + 8 * U)


@pytest.mark.parametrize("T,H", [(305, 8), (3001, 64), (700, 256), (1300, 264), (999, 513), (2100, 1411), (641, 2048),
                                 (457, 4096), (310, 8191), (305, 14336), (306, 16384), (304, 32768)])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("res", [False, True])
def test_norm_many_rows(T, H, dt, res):
    """More rows than CTAs: the persistent kernel, whose grids these T do not divide."""
    rng = gen(T, H, dt, res)
    x = place(rng.standard_normal((T, H), np.float32) * 2, DT[dt])
    w = torch.as_tensor(rng.normal(1, 0.3, H)).to(DT[dt]).cuda()
    r = place(rng.standard_normal((T, H), np.float32) * 3, DT[dt]) if res else None
    s, y = ops.rms_norm(f64(x), f64(w), 1e-5, f64(r) if res else None)
    q = pw.pw_rms_norm_i8(x, w, 1e-5, residual=r, out=(out := torch.empty_like(x)))
    if res:
        check_out(q[2], s, dt, U)
    check_out(out, y, dt, 64 * U, extra=np.abs(f64(w)) * 4 * U if res else 0.0)
    check_q(q[0], q[1], y, 72 * U)
    if not res:
        check_q(*pw.pw_quant_i8(x), f64(x), 2 * U)


@pytest.mark.parametrize("off,pad", [(0, 8), (1, 0), (3, 5), (8, 16)])
@pytest.mark.parametrize("H", [63, 128, 1411, 5000])
def test_norm_strides_and_frames(off, pad, H):
    T = 4
    rng = gen(off, pad, H)
    x = place(rng.normal(0, 1, (T, H)), torch.float16, pad, off)
    r = place(rng.normal(0, 1, (T, H)), torch.float16, pad + 3, off)
    w = torch.as_tensor(rng.normal(1, 0.1, H)).half().cuda()
    y, sm = Framed(T, H, torch.float16, pad, off), Framed(T, H, torch.float16, off, pad)
    q = Framed(T, H, torch.int8, pad, off)
    scale = torch.empty(T, device="cuda")
    pw.pw_rms_norm_i8(x, w, 1e-6, residual=r, q=q.view, scale=scale, out=y.view, sum_out=sm.view)
    s_ref, y_ref = ops.rms_norm(f64(x), f64(w), 1e-6, f64(r))
    check_out(y.view, y_ref, "f16", 64 * U, extra=4 * U * 2)
    check_out(sm.view, s_ref, "f16", U)
    check_q(q.view, scale, y_ref, 72 * U)
    assert y.intact() and sm.intact() and q.intact()


def test_norm_updates_the_residual_in_place():
    rng = gen(9)
    for H in (4096, 1411, 50000):
        x = place(rng.normal(0, 1, (3, H)), torch.bfloat16)
        r = place(rng.normal(0, 1, (3, H)), torch.bfloat16)
        w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
        y1, s1 = pw.pw_rms_norm(x, w, 1e-6, residual=r)
        r2 = r.clone()
        y2, s2 = pw.pw_rms_norm(x, w, 1e-6, residual=r2, sum_out=r2)
        assert torch.equal(y1, y2) and torch.equal(s1, r2) and s2 is r2


def test_norm_rows_of_zeros_and_of_no_numbers():
    x = torch.zeros(5, 256, device="cuda", dtype=torch.float16)
    x[1, 7] = float("nan")
    x[2, 9] = INF
    x[3] = 65504.0
    x[4, 0] = 6e-8
    w = torch.ones(256, device="cuda", dtype=torch.float16)
    q, s, = pw.pw_rms_norm_i8(x, w, 1e-6)
    y = pw.pw_rms_norm(x, w, 1e-6)
    assert (q[0] == 0).all() and s[0] == 0 and (y[0] == 0).all()
    assert torch.isnan(s[1]) and torch.isnan(y[1]).all()
    assert not torch.isfinite(s[2])
    assert (q[3] == 127).all() and torch.isfinite(y[3]).all()
    assert q[4, 0] == 127 and (q[4, 1:] == 0).all()


@pytest.mark.parametrize("T,K", [(1, 1), (3, 17), (2, 512), (5, 1411), (9, 4096), (3, 14336), (1, 70000)])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_quant(T, K, dt):
    rng = gen(T, K, dt)
    x = place(rng.normal(0, 5, (T, K)), DT[dt])
    q, s = pw.pw_quant_i8(x)
    check_q(q, s, f64(x), 2 * U)


@pytest.mark.parametrize("T,K", [(3, 1411), (4, 4096), (2, 14336), (500, 512), (2, 70000)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_quant_of_16_bit_rows_rounds_as_the_quotient_does(T, K, dt):
    # In whole numbers, halves to even.  No tolerance: a quotient 127 a / b of
    # numbers of 11 digits that is no half lies q 2^-19 or more from one, and the
    # kernel's, rounded once from a factor of twice fp32's digits, within q 2^-23.
    rng = gen(T, K, dt, "halves")
    x = rng.normal(0, 5, (T, K))
    x[np.abs(x) < 2.0 ** -6] = 0
    x[0, :K // 2] = rng.integers(-254, 255, K // 2) / 2     # every quotient a whole number or a half
    x[0, 0], x[0, K // 2:] = 127, 0
    x = place(x, DT[dt])
    q, _ = pw.pw_quant_i8(x)
    n = np.round(f64(x) * 2 ** 24).astype(np.int64)         # exact: 2^-24 divides every value
    a = np.abs(n)
    den = 2 * a.max(1, keepdims=True)
    num = 254 * a + den // 2
    want = num // den
    want -= (num % den == 0) & (want % 2 == 1)
    assert (q.cpu().numpy() == np.sign(n) * want).all()


def test_quant_extremes():
    x = torch.zeros(6, 64, device="cuda")
    x[0, 3], x[0, 4] = 1e-38, -0.5e-38          # 127 / max overflows fp32
    x[1] = -0.0
    x[2, 5] = float("nan")
    x[3, 5] = -INF
    x[4, 1], x[4, 2] = 3e38, -3e38
    x[5, :2] = torch.tensor([2.0, -1.0])
    q, s = pw.pw_quant_i8(x)
    assert q[0, 3] == 127 and q[0, 4] in (-63, -64) and (q[1] == 0).all() and s[1] == 0
    assert torch.isnan(s[2]) and (q[2] == 0).all() and s[3] == INF and (q[3] == 0).all()
    assert q[4, 1] == 127 and q[4, 2] == -127 and torch.isfinite(s[4])
    assert q[5, 0] == 127 and q[5, 1] == -64     # -63.5: to the even neighbour


def _i8(rng, T, K):
    """Any int8 in rows padded to 16 bytes, the padding too (it must not count)."""
    raw = torch.as_tensor(rng.integers(-128, 128, (T, (K + 15) // 16 * 16), dtype=np.int8)).cuda()
    return raw[:, :K]


def _linear_case(T, N, K, dt, bias, seed=0):
    rng = gen(T, N, K, dt, bias, seed)
    x, w = _i8(rng, T, K), _i8(rng, N, K)
    xs = torch.as_tensor(rng.uniform(0.001, 0.1, T), dtype=torch.float32).cuda()
    ws = torch.as_tensor(rng.uniform(0.0001, 0.01, N), dtype=torch.float32).cuda()
    b = torch.as_tensor(rng.normal(0, 1, N)).to(DT[dt]).cuda() if bias else None
    return x, xs, w, ws, b


LINEARS = [(1, 1, 1), (1, 8, 16), (1, 60, 2048), (4, 60, 2048), (3, 129, 1411), (2, 1000, 4096), (5, 300, 14336),
           (8, 257, 512), (9, 128, 256), (16, 130, 1023), (17, 300, 1040), (31, 200, 4096), (33, 128, 64),
           (64, 384, 2049), (65, 260, 130), (100, 1411, 1411), (128, 256, 1024), (129, 100, 5000), (255, 513, 96),
           (256, 256, 2048), (257, 640, 1100), (300, 1000, 3000), (700, 90, 16), (1024, 512, 1056)]


@pytest.mark.parametrize("T,N,K", LINEARS)
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_linear(T, N, K, dt):
    x, xs, w, ws, b = _linear_case(T, N, K, dt, (T + N) % 2)
    out = Framed(T, N, DT[dt], pad=T % 3, off=N % 5)
    pw.pw_linear_i8(x, xs, w, ws, bias=b, out=out.view)
    acc, ref = ops.linear_i8(f64(x), f64(xs), f64(w), f64(ws), None if b is None else f64(b))
    # fp16 outputs may overflow for none of these sizes: |acc| <= 2^14 K, scales below 1e-3 together
    lim = 65504.0 if dt == "f16" else 1e38
    fine = np.abs(ref) < lim
    prod = np.abs(acc * f64(xs)[:, None] * f64(ws)[None, :])
    tol = prod * 3 * U + np.abs(ref) * (ROUND[dt] + U) + 2.0 ** -25
    assert (np.abs(f64(out.view) - ref)[fine] <= tol[fine]).all()
    assert out.intact()


@pytest.mark.parametrize("T", [1, 4, 16, 40, 130, 300])
@pytest.mark.parametrize("K", [100, 2000, 16384, 131071])
def test_linear_sums_are_exact(T, K):
    """Rows at the int8 limits: sums up to 2^31, far past what fp32 holds, must
    come out as the correctly rounded fp32 of the exact int32."""
    rng = gen(T, K, "exact")
    N = 40
    x, w = _i8(rng, T, K), _i8(rng, N, K)
    x[0] = -128
    w[0] = -128
    w[1] = 127
    w[2] = -128
    w[2, -1] = 127
    one = lambda n: torch.ones(n, device="cuda")
    got = pw.pw_linear_i8(x, one(T), w, one(N), out_dtype=torch.float32)
    acc = f64(x) @ f64(w).T
    assert np.array_equal(f64(got), acc.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("T", [3, 13, 20, 50, 100, 131, 300, 520])
@pytest.mark.parametrize("N,K", [(20011, 200), (14337, 1040), (9001, 2100), (30000, 70), (77, 1), (300, 3), (1, 65)])
def test_linear_many_channels(T, N, K):
    # tiles of every width and token count; sums below 2^20, exact in fp32
    rng = gen(T, N, K)
    x, w = [torch.as_tensor(rng.integers(-16, 17, (n, (K + 15) // 16 * 16), dtype=np.int8)).cuda()[:, :K] for n in (T, N)]
    one = torch.ones(max(T, N), device="cuda")
    out = torch.full((T, N + 3), -7.0, device="cuda")
    pw.pw_linear_i8(x, one[:T], w, one[:N], out=out[:, 1:N + 1])
    assert torch.equal(out[:, 1:N + 1].double(), x.double() @ w.double().T)
    assert (out[:, 0] == -7).all() and (out[:, N + 1:] == -7).all()


@pytest.mark.parametrize("T,N,K", [(17, 60, 2048), (33, 60, 9000), (64, 520, 1411), (250, 130, 16384), (1000, 57, 70),
                                   (40, 4096, 2100), (70, 1300, 16384), (5000, 40, 300), (100, 3000, 16384),
                                   (64, 4100, 131071), (40, 20011, 5000), (130, 20011, 5000), (300, 1030, 131071),
                                   (300, 2000, 16384)])
def test_linear_sums_are_exact_in_every_kernel(T, N, K):
    """Small and large work by token blocks, few and many tiles, K whole and
    split: the fp32 of the exact sum."""
    rng = gen(T, N, K, "kernels")
    x, w = _i8(rng, T, K), _i8(rng, N, K)
    x[0], w[0], w[N // 2, ::2] = -128, -128, 127
    one = torch.ones(max(T, N), device="cuda")
    out = torch.empty(T, N, device="cuda")
    pw.pw_linear_i8(x, one[:T], w, one[:N], out=out)
    # sums below 2^31 are exact in 64 bits
    assert torch.equal(out, (x.double() @ w.double().T).float())


def test_linear_bf16_and_wide_rows():
    rng = gen(44)
    x, xs, w, ws, b = _linear_case(37, 333, 4096, "bf16", True)
    wide = torch.zeros(333, 4096 + 160, dtype=torch.int8, device="cuda")
    wide[:, 32:32 + 4096] = w
    xw = torch.zeros(37, 4096 + 48, dtype=torch.int8, device="cuda")
    xw[:, 16:16 + 4096] = x
    a = pw.pw_linear_i8(x, xs, w, ws, bias=b, out_dtype=torch.bfloat16)
    c = pw.pw_linear_i8(xw[:, 16:16 + 4096], xs, wide[:, 32:32 + 4096], ws, bias=b, out_dtype=torch.bfloat16)
    assert torch.equal(a, c)
    check_out(a, ops.linear_i8(f64(x), f64(xs), f64(w), f64(ws), f64(b))[1], "bf16", 8 * U, extra=1e-5)


def test_quantised_rows_feed_the_product():
    rng = gen(5)
    x = place(rng.normal(0, 1, (6, 1411)), torch.float16)
    wt = place(rng.normal(0, 0.02, (70, 1411)), torch.float16)
    (q, s), (wq, wsc) = pw.pw_quant_i8(x), pw.pw_quant_i8(wt)
    got = pw.pw_linear_i8(q, s, wq, wsc, out_dtype=torch.float32)
    ref = f64(x) @ f64(wt).T
    # half a step of each side on every term: sqrt(K) * (s/2 |w| + ws/2 |x|) in the 2-norm sense
    assert np.linalg.norm(f64(got) - ref) <= 0.05 * np.linalg.norm(ref)


def _check_logprobs(x, ids, top, got, nan_rows=()):
    ref = ops.logprobs(f64(x), None if ids is None else ids.cpu().numpy(), top)
    V = x.shape[1]
    rel = (V / 256 + 32 + 24) * U
    keep = np.array([t not in nan_rows for t in range(x.shape[0])])

    def near(g, r, scale):
        g, r = f64(g)[keep], r[keep]
        fin = np.isfinite(r)
        assert np.array_equal(g[~fin], r[~fin])
        d = np.abs(g - np.where(fin, r, 0))[fin]
        assert (d <= rel * (1 + scale) + 4 * U * np.abs(r[fin])).all(), d.max()
    near(got.entropy, ref["entropy"], 2 * np.log(V))
    if ids is not None:
        near(got.logprob, ref["logprob"], 1)
        assert np.array_equal(got.rank.cpu().numpy()[keep], ref["rank"][keep])
    if top:
        assert np.array_equal(got.top_ids.cpu().numpy()[keep], ref["top_ids"][keep])
        near(got.top_logprobs, ref["top_logprobs"], 1)


LOGS = [(1, 1, 1), (2, 2, 2), (3, 7, 5), (1, 31, 31), (2, 33, 32), (5, 100, 0), (4, 511, 32), (3, 513, 1),
        (2, 4095, 20), (1, 32000, 5), (3, 50001, 32), (1, 131072, 20), (200, 1000, 3), (700, 777, 32),
        (40, 20011, 8)]


@pytest.mark.parametrize("T,V,top", LOGS)
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_logprobs(T, V, top, dt):
    rng = gen(T, V, top, dt)
    x = place(rng.normal(0, 3, (T, V)), DT[dt], pad=V % 3, off=T % 4)
    ids = torch.as_tensor(rng.integers(0, V, T), dtype=torch.int64 if T % 2 else torch.int32).cuda()
    _check_logprobs(x, ids, top, pw.pw_logprobs(x, ids, top=top))


@pytest.mark.parametrize("off", range(9))
@pytest.mark.parametrize("V", [5, 300, 9001])
def test_logprobs_rows_start_anywhere(off, V):
    rng = gen(off, V)
    x = place(rng.normal(0, 2, (3, V)), torch.float16, pad=off % 4, off=off)
    ids = torch.tensor([0, V - 1, V // 2], device="cuda")
    _check_logprobs(x, ids, 5, pw.pw_logprobs(x, ids, top=5))


@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "two_values", "steps", "one_left", "lowest",
                                  "lowest_mask", "signed_zeros", "far", "large", "huge", "masks"])
@pytest.mark.parametrize("V", [40, 3001, 70000])
@pytest.mark.parametrize("T", [1, 170])
def test_logprobs_orders_ties_and_masks(kind, V, T):
    rng = gen(kind, V)
    k = np.arange(V)
    row = {"equal": np.full(V, 1.5), "ascending": k * 0.25, "descending": -k * 0.25,
           "two_values": rng.integers(0, 2, V) * 1.0, "steps": (k // 7) % 50 * 1.0,
           "one_left": np.where(k == V // 3, 2.0, -INF), "lowest": np.full(V, float(np.finfo(np.float32).min)),
           "lowest_mask": np.where(k % 3 == 0, rng.normal(0, 1, V), float(np.finfo(np.float32).min)),
           "signed_zeros": np.where(k % 2 == 0, -0.0, 0.0),
           "far": np.where(k == 5, 1e4, -1e4), "large": rng.normal(0, 2, V) + 3e6, "huge": rng.normal(0, 1, V) * 1e30,
           "masks": rng.choice([-1e4, -1e9, -1e30, -INF, 0.5, -2.0], V)}[kind]
    x = place(np.repeat(row[None].astype(np.float32), T, 0), torch.float32)
    ids = torch.as_tensor(rng.integers(0, V, T)).cuda()
    top = 32
    _check_logprobs(x, ids, top, pw.pw_logprobs(x, ids, top=top))


@pytest.mark.parametrize("V", [33, 5000, 140000])
def test_logprobs_rows_of_nothing_and_of_no_numbers(V):
    rng = gen(V, "nan")
    a = rng.normal(0, 1, (7, V)).astype(np.float32)
    a[0] = -INF
    a[1, 3] = np.nan
    a[2, 4] = INF
    a[3, 5:] = -INF
    a[4] = np.nan
    a[6, :] = -INF
    x = place(a, torch.float32)
    ids = torch.tensor([2, 3, 4, 6, 0, -1, V], device="cuda")
    g = pw.pw_logprobs(x, ids, top=6)
    keep = (1, 2, 4)
    _check_logprobs(x, ids, 6, g, nan_rows=keep)
    for t in keep:
        assert torch.isnan(g.logprob[t]) and torch.isnan(g.entropy[t]) and torch.isnan(g.top_logprobs[t]).all()
    assert 3 not in g.top_ids[1].tolist() and (g.top_ids[4] == -1).all() and g.top_ids[2, 0] == 4
    assert g.rank[1] == -1 and g.rank[4] == -1 and g.rank[2] == 0


def test_logprobs_parts():
    x = place(gen(3).normal(0, 1, (4, 999)), torch.bfloat16)
    ids = torch.tensor([1, 2, 3, 4], device="cuda", dtype=torch.int32)
    a = pw.pw_logprobs(x, ids, top=7)
    b = pw.pw_logprobs(x)
    assert b.logprob is None and b.rank is None and torch.equal(a.entropy, b.entropy)
    out = pw.LogProbs(torch.empty(4, device="cuda"), None, None, None, None)
    c = pw.pw_logprobs(x, ids, out=out)
    assert torch.equal(c.logprob, a.logprob) and c.logprob is out.logprob


def _all_calls(st):
    y, s = pw.pw_rms_norm(st["x"], st["w"], residual=st["r"])
    q, sc, _ = pw.pw_rms_norm_i8(st["x"], st["w"], residual=st["r"])
    q2, s2 = pw.pw_quant_i8(y)
    z = [pw.pw_linear_i8(q, sc, st["wq"], st["ws"], out_dtype=torch.float32), pw.pw_linear_i8(q2, s2, st["wq"], st["ws"])]
    lp = pw.pw_logprobs(z[0], st["ids"], top=9)
    return [y, s, q, sc, q2, s2, *z, *lp]


def _state(T):
    rng = gen(T, "state")
    wt = place(rng.normal(0, 0.1, (5001, 1024)), torch.float16)
    wq, ws = pw.pw_quant_i8(wt)
    return dict(x=place(rng.normal(0, 1, (T, 1024)), torch.float16), r=place(rng.normal(0, 1, (T, 1024)), torch.float16),
                w=torch.ones(1024, dtype=torch.float16, device="cuda"), wq=wq, ws=ws,
                ids=torch.as_tensor(rng.integers(0, 5001, T)).cuda())


@pytest.mark.parametrize("T", [1, 8, 50, 400])
def test_same_bits_again_on_other_streams_and_in_a_graph(T):
    st = _state(T)
    a = _all_calls(st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = _all_calls(st)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = _all_calls(st)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for u, v, w in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, w)


def test_offsets_past_31_bits():
    """Rows far apart: the third row starts past 2^31 elements."""
    ld = (1 << 30) + 64
    base = torch.zeros(2 * ld + 4096, dtype=torch.float16, device="cuda")
    x = base.as_strided((3, 4096), (ld, 1))
    rng = gen("far")
    x.copy_(torch.as_tensor(rng.normal(0, 1, (3, 4096))))
    near = x.contiguous()
    w = torch.ones(4096, dtype=torch.float16, device="cuda")
    assert torch.equal(pw.pw_rms_norm(x, w), pw.pw_rms_norm(near, w))
    ids = torch.tensor([5, 6, 7], device="cuda")
    for u, v in zip(pw.pw_logprobs(x, ids, top=4), pw.pw_logprobs(near, ids, top=4)):
        assert torch.equal(u, v)
    q, s = pw.pw_quant_i8(near)
    b8 = base.view(torch.int8)
    far = b8.as_strided((3, 4096), (ld, 1))
    far.copy_(q)
    ones = torch.ones(3, device="cuda")
    ref = f64(q) @ f64(q).T
    for T in (3, 1):
        got = pw.pw_linear_i8(far[:T], ones[:T], far, ones, out_dtype=torch.float32)
        assert np.array_equal(f64(got), ref[:T])
    big = torch.as_tensor(rng.integers(-127, 128, (40, 4096), dtype=np.int8)).cuda()
    got = pw.pw_linear_i8(big, torch.ones(40, device="cuda"), far, ones, out_dtype=torch.float32)
    assert np.array_equal(f64(got), f64(big) @ f64(q).T)


def test_linear_waits_have_all_ended():
    assert pw.pw_linear_i8_status() == 0
