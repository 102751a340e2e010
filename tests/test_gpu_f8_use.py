"""The operators of an 8-bit expert layer as programs use them: in a decode step, on
several streams at once, in graphs that share nothing, with rows far apart, experts that
share weights, and the status of bounded waits."""
import os
import sys

import numpy as np
import pytest
import torch

import any_precision_weight_gb300 as pw
import synth
from oracle import f8

from test_gpu_f8 import F8, cuda, near, product_tol, scales, values
from test_gpu_operators import U, f64, gen

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def check(out, x, xs, w, ws, dt="f32"):
    ref, size = f8.linear(f64(x), f64(xs), f64(w), f64(ws))
    near(out, ref, dt, product_tol(size, x.shape[1], dt) + 2 * U * np.abs(ref))


@pytest.mark.parametrize("batch", [1, 5, 20, 100])
def test_a_decode_step_with_8_bit_experts(batch):
    from decode_step import DecodeStep
    cfg = synth.CONFIGS["tiny"]
    m = DecodeStep(cfg, batch, 2, 3001, experts="f8")
    x = torch.from_numpy(synth.tokens(cfg, T=batch)).cuda()
    ids = torch.as_tensor(np.random.default_rng(batch).integers(0, 3001, batch)).cuda()
    trace = []
    want = m.step(x, ids, trace=trace)
    for _, l, y, logits, shared, out in [t for t in trace if t[0] == "moe"]:
        e = m.f8[l]
        r = f8.route(f64(logits), cfg.top_k, cfg.renorm)
        ref = f64(shared)
        # the whole layer in 64 bits, roundings between its stages left out: two quantisations
        # of 2^-4 and two products rounded to fp16 change it by a few hundredths
        up = f64(e.gate_up) * np.stack([f8.spread(s, f8.B, *e.gate_up.shape[1:]) for s in f64(e.gate_up_scale)])
        down = f64(e.down) * np.stack([f8.spread(s, f8.B, *e.down.shape[1:]) for s in f64(e.down_scale)])
        mix = np.zeros_like(ref)
        for t in range(batch):
            for j, k in enumerate(r["idx"][t]):
                mix[t] += r["weight"][t, j] * (down[k] @ f8.silu_up((up[k] @ f64(y)[t])[None])[0])
        got = f64(out) - ref
        assert np.linalg.norm(got - mix) <= 0.06 * np.linalg.norm(mix)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = m.step(x, ids)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert pw.pw_linear_f8_status() == 0


@pytest.mark.parametrize("T", [3, 60, 400])
def test_products_on_several_streams_at_once(T):
    rng = gen(T, "streams")
    K, N = 1000, 1500
    sets = [(values(rng, T, K), scales(rng, T, 8), values(rng, N, K), scales(rng, 12, 8)) for _ in range(4)]
    want = [pw.pw_linear_f8(*s, out_dtype=torch.float32) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[pw.pw_linear_f8(*s, out_dtype=torch.float32, stream=st) for s, st in zip(sets, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, want):
            assert torch.equal(a, b)   # a repeated call gives the same bits
    assert pw.pw_linear_f8_status() == 0


def test_two_graphs_of_routing_and_products():
    """Each capture has memory of its own: replays in any order, and eager calls between them."""
    from any_precision_weight_gb300.model import F8Experts
    rng = gen(9, "graphs")
    m = F8Experts(cuda(rng.normal(0, 0.06, (8, 512, 256)), torch.float16), cuda(rng.normal(0, 0.06, (8, 256, 256)), torch.float16))
    ins = [(cuda(rng.normal(0, 1, (T, 256)), torch.float16), cuda(rng.normal(0, 1, (T, 8)), torch.float32)) for T in (7, 300)]
    want = [m.forward(x, l, 2, True) for x, l in ins]
    torch.cuda.synchronize()
    graphs = []
    for x, l in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = m.forward(x, l, 2, True)
        graphs.append((g, out))
    for i in (0, 1, 1, 0, 0, 1):
        graphs[i][0].replay()
        again = m.forward(*ins[1 - i], 2, True)
        torch.cuda.synchronize()
        assert torch.equal(graphs[i][1], want[i]) and torch.equal(again, want[1 - i])


@pytest.mark.parametrize("T", [4, 40, 200])
def test_rows_far_apart(T):
    """Offsets past 32 bits: rows of x and out, experts' weights."""
    rng = gen(T, "far")
    K, N, far = 384, 320, (1 << 33) // T // 16 * 16
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB of the GPU's memory")
    x = torch.zeros(far * (T - 1) + K, dtype=torch.uint8, device="cuda").view(F8).as_strided((T, K), (far, 1))
    x.copy_(values(rng, T, K))
    xs, ws = scales(rng, T, 3), scales(rng, 2, 3, 3)
    apart = (1 << 32) + 4096
    w = torch.zeros(apart + N * K, dtype=torch.uint8, device="cuda").view(F8).as_strided((2, N, K), (apart, K, 1))
    w.copy_(values(rng, 2, N, K))
    out = torch.zeros(far * (T - 1) + N, dtype=torch.float16, device="cuda").as_strided((T, N), (far, 1))
    xs *= 2.0 ** -14
    n = T // 3
    pw.pw_grouped_linear_f8(x, xs, w, ws, cuda(np.array([0, n, T]), torch.int32), out=out)
    check(out[:n], x[:n], xs[:n], w[0], ws[0], "f16")
    check(out[n:], x[n:], xs[n:], w[1], ws[1], "f16")
    pw.pw_linear_f8(x, xs, w[1], ws[1], out=out)
    check(out, x, xs, w[1], ws[1], "f16")
    h = torch.zeros(far * (T - 1) + K, dtype=torch.float16, device="cuda").as_strided((T, K), (far, 1))
    h.copy_(cuda(rng.normal(0, 1, (T, K)), torch.float16))
    q, s = pw.pw_quant_f8(h, q=x)
    v, ref = f8.quotients(f64(h))
    assert np.array_equal(f64(q), f8.e4m3(v)) and (np.abs(f64(s) - ref) <= ref * U).all()
    back = np.arange(T)[::-1].copy()
    got = pw.pw_combine(h, torch.ones(T, 1, device="cuda"), cuda(back, torch.int32), residual=h[:, :K])
    near(got, f64(h)[back] + f64(h), "f16", 0)


@pytest.mark.parametrize("T", [5, 100, 900])
def test_experts_that_share_weights(T):
    rng = gen(T, "shared")
    K, N, E = 256, 300, 3
    x, xs, w, ws = values(rng, T, K), scales(rng, T, 2), values(rng, N, K), scales(rng, 3, 2)
    off = cuda(np.array([0, T // 4, T // 2, T]), torch.int32)
    got = pw.pw_grouped_linear_f8(x, xs, w[None].expand(E, N, K), ws[None].expand(E, 3, 2), off, out_dtype=torch.float32)
    check(got, x, xs, w, ws)


@pytest.mark.parametrize("T,N,K", [(1, 28672, 4096), (40, 4096, 14336), (130, 1030, 520), (600, 2100, 1411)])
def test_scales_of_any_stride(T, N, K):
    rng = gen(T, N, "strides")
    kb, nb = f8.blocks(K), f8.blocks(N)
    x, w = values(rng, T, K), values(rng, N, K)
    xs, ws = scales(rng, T, kb + 3)[:, 2:2 + kb], scales(rng, nb, kb + 5)[:, 1:1 + kb]
    a = pw.pw_linear_f8(x, xs, w, ws, out_dtype=torch.float32)
    assert torch.equal(a, pw.pw_linear_f8(x, xs.contiguous(), w, ws.contiguous(), out_dtype=torch.float32))
    check(a[:, :500], x, xs, w[:500], ws[:4])


def test_status_tells_once():
    assert pw.pw_linear_f8_status() == 0
    pw.pw_debug_linear_f8_timeout()
    assert pw.pw_linear_f8_status() == pw.PW_STATUS_TIMEOUT
    assert pw.pw_linear_f8_status() == 0 and pw.pw_linear_i8_status() == 0
