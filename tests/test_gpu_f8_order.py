"""Calls in a row on one stream, some of which begin before the one ahead has ended.

pw_moe_forward of a few tokens reads the logits and the blocks' descriptors before it waits for
the kernel ahead of it; pw_quant_f8, pw_silu_quant_f8 and pw_route let the next kernel begin as
soon as all before them has ended.  Whatever wrote the logits has then ended too.  Each sequence
gives the bits that it gives with a wait of the host behind every call.
"""
import numpy as np
import pytest
import torch

import any_precision_weight_gb300 as pw
import synth
from _layers import LIVE
from any_precision_weight_gb300.model import F8Experts, load_expert_layer

from test_gpu_f8 import cuda, scales, values
from test_gpu_operators import gen

pytestmark = pytest.mark.gpu

CFG = synth.CONFIGS["tiny"]
STEPS = 30


@pytest.fixture(scope="module")
def layer():
    m = pw.PagedMoE(1, CFG.E, CFG.H, CFG.I, guard=256)
    load_expert_layer(m, 0, lambda e, kind: (synth.parent_indices(CFG, 0, e, kind), synth.parent_lut(CFG, 0, e, kind)),
                      synth.block_bits(CFG))
    return m


class Between:
    """What runs between the logits and the layer, long enough for the layer to begin beside it."""

    def __init__(self, rng, T):
        self.wide = cuda(rng.normal(0, 1, (8192, 4096)), torch.float16)
        self.up = cuda(rng.normal(0, 1, (2048, 8192)), torch.float16)
        self.many = cuda(rng.normal(0, 1, (8192, CFG.E)), torch.float32)
        self.rows = cuda(rng.integers(0, 8192, 8192), torch.int32)

    def quant(self, logits, perm):
        return pw.pw_quant_f8(self.wide)

    def gathered(self, logits, perm):
        return pw.pw_quant_f8(self.wide, rows=self.rows)

    def silu(self, logits, perm):
        return pw.pw_silu_quant_f8(self.up)

    def routes(self, logits, perm):   # the same logits, and many others
        return (*pw.pw_route(logits, CFG.top_k, CFG.renorm), *pw.pw_route(self.many, CFG.top_k))

    def all_of_them(self, logits, perm):
        return (*self.routes(logits, perm), *self.quant(logits, perm), *pw.pw_route(logits, CFG.top_k))

    def tokens_of_the_layer_before(self, logits, perm):
        """Gathered by the order that the layer's last call wrote."""
        return pw.pw_quant_f8(self.wide, rows=perm, per=CFG.top_k)


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.dtype is torch.float8_e4m3fn else x,
                           y.view(torch.uint8) if y.dtype is torch.float8_e4m3fn else y) for x, y in zip(a, b))


@pytest.mark.parametrize("T", [1, 4, 40])
@pytest.mark.parametrize("what", ["quant", "gathered", "silu", "routes", "all_of_them", "tokens_of_the_layer_before"])
def test_logits_written_then_an_early_kernel_then_the_layer(layer, T, what):
    LIVE.append(layer)
    rng = gen(T, what, "order")
    mid = getattr(Between(rng, T), what)
    x = torch.from_numpy(synth.tokens(CFG, T=T)).cuda()
    new = cuda(rng.normal(0, 2, (STEPS, T, CFG.E)), torch.float32)
    ws = layer.workspace(T, CFG.top_k)

    def run(wait):
        logits, perm, outs = torch.zeros_like(new[0]), torch.zeros(T * CFG.top_k, dtype=torch.int32, device="cuda"), []
        wait()
        for i in range(STEPS):
            logits.copy_(new[i])
            wait()
            made = mid(logits, perm)
            wait()
            o = layer.pw_moe_forward(0, x, logits, CFG.top_k, CFG.renorm, ws=ws, routing=True)
            perm = o[4]
            wait()
            outs.append((*made, *o))
        torch.cuda.synchronize()
        return outs

    want, got = run(torch.cuda.synchronize), run(lambda: None)
    for a, b in zip(want, got):
        assert _same(a, b)
    assert layer.workspace_status(ws) == 0


@pytest.mark.parametrize("T", [1, 4, 40])
@pytest.mark.parametrize("way", [None, (0, 8, 1, 4), (0, 16, 2, 1), (1, 64, 64, 1), (1, 128, 64, 4), (2, 128, 128, 2)])
def test_logits_of_an_8_bit_product(layer, T, way):
    """The router as pw_linear_f8 in fp32, right ahead of the layer."""
    LIVE.append(layer)
    rng = gen(T, *(way or ()), "router")
    K = 4096
    x = torch.from_numpy(synth.tokens(CFG, T=T)).cuda()
    w, ws = values(rng, CFG.E, K), scales(rng, 1, K // 128)
    ins = [cuda(rng.normal(0, 1, (T, K)), torch.float16) for _ in range(STEPS)]
    logits = torch.zeros(T, CFG.E, device="cuda")
    space = layer.workspace(T, CFG.top_k)

    def run(wait):
        outs = []
        for h in ins:
            q, s = pw.pw_quant_f8(h)
            s = s * 2.0 ** -12
            wait()
            if way:
                pw.pw_debug_linear_f8(way, q, s, w[None], ws[None], out=logits)
            else:
                pw.pw_linear_f8(q, s, w, ws, out=logits)
            wait()
            outs.append(layer.pw_moe_forward(0, x, logits, CFG.top_k, CFG.renorm, ws=space, routing=True))
            wait()
        torch.cuda.synchronize()
        return outs

    want, got = run(torch.cuda.synchronize), run(lambda: None)
    for a, b in zip(want, got):
        assert _same(a, b)


def test_both_kinds_of_experts_in_turn_eagerly_and_as_a_graph(layer):
    """A step of logits, 8-bit experts, planes, quantiser and planes again; replays get other inputs."""
    LIVE.append(layer)
    rng = gen(5, "both")
    T = 6
    f8 = F8Experts(cuda(rng.normal(0, CFG.H ** -0.5, (CFG.E, 2 * CFG.I, CFG.H)), torch.float16),
                   cuda(rng.normal(0, CFG.I ** -0.5, (CFG.E, CFG.H, CFG.I)), torch.float16))
    wide = cuda(rng.normal(0, 1, (4096, 4096)), torch.float16)
    xs = [torch.from_numpy(synth.tokens(CFG, T=T)).cuda() * (0.2 * (i + 1)) for i in range(8)]
    new = cuda(rng.normal(0, 2, (8, T, CFG.E)), torch.float32)
    x, source, logits = torch.zeros_like(xs[0]), torch.zeros_like(new[0]), torch.zeros_like(new[0])
    ws = layer.workspace(T, CFG.top_k)

    def step(wait):
        logits.copy_(source)
        wait()
        a = f8.forward(x, logits, CFG.top_k, CFG.renorm)
        wait()
        b = layer.pw_moe_forward(0, a, logits, CFG.top_k, CFG.renorm, residual=x, ws=ws)
        wait()
        logits.neg_()
        wait()
        q, s = pw.pw_quant_f8(wide)
        wait()
        c = layer.pw_moe_forward(0, b, logits, CFG.top_k, CFG.renorm, ws=ws)
        wait()
        return a, b, c, q, s

    def inputs(i):
        x.copy_(xs[i])
        source.copy_(new[i])

    want = []
    for i in range(8):
        inputs(i)
        want.append([o.clone() for o in step(torch.cuda.synchronize)])
    for i in range(8):
        inputs(i)
        assert _same(step(lambda: None), want[i])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(lambda: None)
    for i in (3, 0, 7, 7, 1, 2):
        inputs(i)
        g.replay()
        torch.cuda.synchronize()
        assert _same(outs, want[i])
    assert pw.pw_linear_f8_status() == 0 and layer.workspace_status(ws) == 0
