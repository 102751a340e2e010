"""The operators and the expert layer in one decode step (examples/decode_step.py):
every call against the oracle on what it read, and the step as a CUDA graph."""
import os
import sys

import numpy as np
import pytest
import torch

import any_precision_weight_gb300 as pw
import synth
from oracle import moe as omoe
from oracle import operators as ops

from _layers import LIVE, SynthBlocks, assert_close, oracle_blocks, to_np
from test_gpu_operators import U, _check_logprobs, check_out, check_q, f64

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def _model(batch):
    from decode_step import DecodeStep
    cfg = synth.CONFIGS["tiny"]
    m = DecodeStep(cfg, batch, 2, 3001, guard=256)
    LIVE.append(m.moe)
    x = torch.from_numpy(synth.tokens(cfg, T=batch)).cuda()
    ids = torch.as_tensor(np.random.default_rng(batch).integers(0, 3001, batch)).cuda()
    return cfg, m, x, ids


@pytest.mark.parametrize("batch", [1, 5, 20, 100])
def test_every_call_of_a_step(batch):
    cfg, m, x, ids = _model(batch)
    trace = []
    m.step(x, ids, trace=trace)
    names = [t[0] for t in trace]
    assert names == ["norm", "linear", "linear", "quant", "linear", "moe"] * 2 + ["norm", "linear", "logprobs"]
    for t in trace:
        if t[0] == "norm":
            _, d, r, w, y, q, s, new = t
            sr, yr = ops.rms_norm(f64(d), f64(w), 1e-6, f64(r))
            check_out(new, sr, "f16", U)
            check_q(q, s, yr, 72 * U)
            if y is not None:
                check_out(y, yr, "f16", 64 * U, extra=8 * U)
        elif t[0] == "quant":
            check_q(t[2], t[3], f64(t[1]), 2 * U)
        elif t[0] == "linear":
            _, q, s, (w, ws), out = t
            acc, ref = ops.linear_i8(f64(q), f64(s), f64(w), f64(ws))
            check_out(out, ref, "f32" if out.dtype == torch.float32 else "f16", 4 * U)
        elif t[0] == "moe":
            _, l, y, logits, shared, out = t
            blocks = oracle_blocks(SynthBlocks(cfg, l), synth.block_bits(cfg, l))
            ref = omoe.layer(to_np(y), to_np(logits), cfg.top_k, cfg.renorm, blocks)
            assert_close(f64(out), ref["out"] + f64(shared))
        else:
            _check_logprobs(t[1], t[2], t[3], t[4])
    assert m.moe.workspace_status(m.ws) == 0 and pw.pw_linear_i8_status() == 0


@pytest.mark.parametrize("batch", [1, 40])
def test_step_as_a_graph(batch):
    cfg, m, x, ids = _model(batch)
    a = m.step(x, ids)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b = m.step(x, ids)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for u, v in zip(a, b):
        assert torch.equal(u, v)
