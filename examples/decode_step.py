"""A decode step around the expert layers: seeded weights, no checkpoint.

Per layer: norm with the residual's addition (int8 and fp16 output), router
product, mixed-precision expert layer (or, with --experts f8, one of e4m3 weights
with a scale for each 128 x 128 block), and a shared expert of dense int8 weights;
then the final norm, the head product and the log probabilities of the tokens that
were chosen, with their alternatives.

    python examples/decode_step.py [--config tiny] [--batch 4] [--layers 2] [--vocab 32000] [--experts planes]

The step is captured into a CUDA graph and replayed; the last replay's tokens
and log probabilities are printed.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import any_precision_weight_gb300 as pw
import synth
from any_precision_weight_gb300.model import F8Experts, load_expert_layer

EPS = 1e-6


def dense(gen, n, k):
    """Seeded dense weights [n][k] as int8 rows with a scale per channel."""
    w = torch.randn(n, k, device="cuda", generator=gen) * k ** -0.5
    return pw.pw_quant_i8(w)


class DecodeStep:
    """Weights and buffers of a small model, and one step over a batch."""

    def __init__(self, cfg, batch: int, n_layers: int, vocab: int, top: int = 5, guard: int = 0,
                 experts: str = "planes"):
        self.cfg, self.T, self.L, self.vocab, self.top = cfg, batch, n_layers, vocab, top
        H, E, S = cfg.H, cfg.E, 2 * cfg.H
        gen = torch.Generator(device="cuda").manual_seed(cfg.seed)
        self.moe = pw.PagedMoE(n_layers, E, H, cfg.I, guard=guard) if experts == "planes" else None
        for l in range(n_layers if self.moe else 0):
            src = lambda e, kind, l=l: (synth.parent_indices(cfg, l, e, kind), synth.parent_lut(cfg, l, e, kind))
            load_expert_layer(self.moe, l, src, synth.block_bits(cfg, l))
        norm = lambda: (1 + 0.1 * torch.randn(H, device="cuda", generator=gen)).half()
        self.norms = [norm() for _ in range(n_layers + 1)]
        self.router = [dense(gen, E, H) for _ in range(n_layers)]
        self.shared_up = [dense(gen, 2 * S, H) for _ in range(n_layers)]       # gate rows, then up rows
        self.shared_down = [dense(gen, H, S) for _ in range(n_layers)]
        self.head = dense(gen, vocab, H)
        self.ws = self.moe.workspace(batch, cfg.top_k) if self.moe else None
        weights = lambda n, k: (torch.randn(E, n, k, device="cuda", generator=gen) * k ** -0.5).half()
        self.f8 = None if self.moe else [F8Experts(weights(2 * cfg.I, H), weights(H, cfg.I)) for _ in range(n_layers)]

    def step(self, x, ids, trace=None):
        """x [T][H] fp16: the batch's residual stream.  ids [T]: the tokens to
        score.  Returns a LogProbs; trace collects what each call read and wrote."""
        note = (lambda *a: None) if trace is None else (lambda *a: trace.append(a))
        delta, stream = torch.zeros_like(x), x
        for l in range(self.L):
            y = torch.empty_like(x)
            q, s, new = pw.pw_rms_norm_i8(delta, self.norms[l], EPS, residual=stream, out=y)
            note("norm", delta, stream, self.norms[l], y, q, s, new)
            logits = pw.pw_linear_i8(q, s, *self.router[l], out_dtype=torch.float32)
            note("linear", q, s, self.router[l], logits)
            up = pw.pw_linear_i8(q, s, *self.shared_up[l])
            note("linear", q, s, self.shared_up[l], up)
            gate, up = up.chunk(2, dim=1)
            act = torch.nn.functional.silu(gate.float()) * up.float()
            aq, asc = pw.pw_quant_i8(act)
            note("quant", act, aq, asc)
            shared = pw.pw_linear_i8(aq, asc, *self.shared_down[l])
            note("linear", aq, asc, self.shared_down[l], shared)
            # the experts' output on top of the shared expert's
            if self.moe:
                delta = self.moe.pw_moe_forward(l, y, logits, self.cfg.top_k, self.cfg.renorm, residual=shared, ws=self.ws)
            else:
                delta = self.f8[l].forward(y, logits, self.cfg.top_k, self.cfg.renorm, residual=shared)
            note("moe", l, y, logits, shared, delta)
            stream = new
        q, s, new = pw.pw_rms_norm_i8(delta, self.norms[self.L], EPS, residual=stream)
        note("norm", delta, stream, self.norms[self.L], None, q, s, new)
        logits = pw.pw_linear_i8(q, s, *self.head, out_dtype=torch.float32)
        note("linear", q, s, self.head, logits)
        out = pw.pw_logprobs(logits, ids, top=self.top)
        note("logprobs", logits, ids, self.top, out)
        return out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--config", default="tiny", choices=sorted(synth.CONFIGS))
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--experts", default="planes", choices=["planes", "f8"])
    a = ap.parse_args()
    m = DecodeStep(synth.CONFIGS[a.config], a.batch, a.layers, a.vocab, experts=a.experts)
    x = torch.from_numpy(synth.tokens(m.cfg, T=a.batch)).cuda()
    ids = torch.arange(a.batch, device="cuda", dtype=torch.int32)
    m.step(x, ids)   # what is set up once per device is set up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.step(x, ids)
    t = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    print(f"{a.config}: {(time.perf_counter() - t) / a.steps * 1e6:.1f} us a step ({a.batch} tokens, {a.layers} layers)")
    for i in range(a.batch):
        alt = ", ".join(f"{k}: {v:.3f}" for k, v in zip(out.top_ids[i].tolist(), out.top_logprobs[i].tolist()))
        print(f"token {int(ids[i])}: logprob {out.logprob[i]:.3f}, rank {int(out.rank[i])}, "
              f"entropy {out.entropy[i]:.3f}; {alt}")
    assert m.moe is None or m.moe.workspace_status(m.ws) == 0
    assert pw.pw_linear_i8_status() == 0 and pw.pw_linear_f8_status() == 0


if __name__ == "__main__":
    main()
