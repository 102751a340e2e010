"""Cases of the operators around the expert layer, for timing and comparison.

Each case is one call of one operator on seeded inputs: the norm with the
residual's addition (pw_rms_norm), the row quantiser (pw_quant_i8), the int8
product (pw_linear_i8) and the log probabilities (pw_logprobs).  ``run``
computes it in plain torch operations in 32 bits, or, where ``own`` is true,
by the framework's entry points; ``exact`` restates it in 64 bits.
"""
from __future__ import annotations

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one sequence's decode step: the norm in front of an expert layer of hidden size 4096
        dict(name="norm_step", op="norm", T=1, H=4096, dtype="f16", residual=True, i8=False),
        # a long prompt batch: the norm that feeds an int8 product, residual stream updated
        dict(name="norm_i8_prefill", op="norm", T=8192, H=4096, dtype="f16", residual=True, i8=True),
        # activations that no norm made, odd sizes: rows of 1411 in a ragged batch
        dict(name="quant_odd", op="quant", T=333, K=1411, dtype="bf16"),
        # a dense weight matrix of the larger layer shape quantised by channel at load time
        dict(name="quant_weights", op="quant", T=28672, K=4096, dtype="f16"),
        # router of the 60-expert layer shape at decode batch 4: the smallest product, latency only
        dict(name="linear_router", op="linear", T=4, N=60, K=2048, out="f32", bias=False),
        # one sequence's decode step through a wide projection: weights stream once
        dict(name="linear_step", op="linear", T=1, N=28672, K=4096, out="f16", bias=False),
        # head over a large vocabulary at a serving batch of 16, logits kept in 32 bits
        dict(name="linear_head", op="linear", T=16, N=131072, K=4096, out="f32", bias=False),
        # ragged batch and odd sizes, with a bias
        dict(name="linear_ragged", op="linear", T=333, N=5003, K=1411, out="bf16", bias=True),
        # the prefill batch through the long-K projection: tensor bound
        dict(name="linear_prefill", op="linear", T=2048, N=4096, K=14336, out="f16", bias=False),
        # one sampled token: its log probability and five alternatives
        dict(name="logprobs_step", op="logprobs", T=1, V=131072, dtype="f32", top=5, masked=False),
        # a small batch under a constrained-decoding mask, odd vocabulary
        dict(name="logprobs_masked", op="logprobs", T=33, V=50001, dtype="f16", top=32, masked=True),
        # scoring a prompt of 2048 given tokens, 20 alternatives each
        dict(name="logprobs_prompt", op="logprobs", T=2048, V=131072, dtype="bf16", top=20, masked=False),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm; odd ones and round ones."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    r = rng.random()
    if r < 0.4:
        v |= 1
    elif r < 0.7 and v >= 64:
        v = v // 32 * 32
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "quant", "linear", "linear", "logprobs"])
    if op == "norm":
        H = _log(rng, 64, 14336)
        T = _log(rng, 1, max(1, min(8192, 8192 * 4096 // H)))
        return dict(op=op, T=T, H=H, dtype=rng.choice(["f16", "bf16"]), residual=rng.random() < 0.7,
                    i8=rng.random() < 0.6)
    if op == "quant":
        K = _log(rng, 64, 14336)
        T = _log(rng, 1, max(1, min(28672, 28672 * 4096 // K)))
        return dict(op=op, T=T, K=K, dtype=rng.choice(["f16", "bf16", "f32"]))
    if op == "linear":
        K = _log(rng, 64, 14336)
        N = _log(rng, 8, min(131072, 131072 * 4096 // K))
        T = _log(rng, 1, max(1, min(2048, 2048 * 4096 * 14336 // (N * K), (1 << 28) // N)))
        return dict(op=op, T=T, N=N, K=K, out=rng.choice(["f16", "bf16", "f32"]), bias=rng.random() < 0.3)
    V = _log(rng, 1000, 152000)
    T = _log(rng, 1, min(2048, 2048 * 131072 // V))
    return dict(op=op, T=T, V=V, dtype=rng.choice(["f16", "bf16", "f32"]), top=rng.choice([0, 1, 5, 20, 32]),
                masked=rng.random() < 0.3)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _rows_i8(T, K):
    """int8 rows that start on 16-byte boundaries, as the quantiser lays them out."""
    return torch.empty(T, (K + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :K]


def _activations(g, T, K):
    """Hidden states as models have them: normal, a hundredth of the channels much larger."""
    x = _normal(g, T, K)
    big = 1.0 + 15.0 * (torch.rand(K, device="cuda", generator=g) < 0.01)
    return x.mul_(big)


def _values_i8(x):
    """(int8 rows, scales) of float rows: inputs that are int8 from the start."""
    s = (x.abs().amax(1, keepdim=True) / 127).clamp_(min=1e-12)
    q = _rows_i8(*x.shape)
    q.copy_((x / s).round_().clamp_(-127, 127))
    return q, s.squeeze(1)


def prepare(case, seed):
    g = _gen(seed)
    op, T = case["op"], case["T"]
    st = {"case": case}
    f32 = dict(dtype=torch.float32, device="cuda")
    if op == "norm":
        H, dt = case["H"], _DT[case["dtype"]]
        st["x"] = _activations(g, T, H).to(dt)
        st["w"] = (1.0 + 0.1 * _normal(g, H)).to(dt)
        st["res"] = (2.0 * _activations(g, T, H)).to(dt) if case["residual"] else None
        st["sum"] = torch.empty(T, H, dtype=dt, device="cuda") if case["residual"] else None
        st["y"] = torch.empty(T, H, dtype=dt, device="cuda")
        if case["i8"]:
            st["q"], st["scale"] = _rows_i8(T, H), torch.empty(T, **f32)
    elif op == "quant":
        K = case["K"]
        st["x"] = _activations(g, T, K).to(_DT[case["dtype"]])
        st["q"], st["scale"] = _rows_i8(T, K), torch.empty(T, **f32)
        # 8-bit results are compared as the values they stand for, held in 16 bits
        st["y"] = torch.empty(T, K, dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float16, device="cuda")
    elif op == "linear":
        N, K = case["N"], case["K"]
        st["x"], st["xs"] = _values_i8(_activations(g, T, K))
        w = _rows_i8(N, K)
        for i in range(0, N, 16384):  # weights: the integers of normal rows, a few at the limits
            n = min(16384, N - i)
            w[i:i + n].copy_(_normal(g, n, K).mul_(36.0).round_().clamp_(-127, 127))
        st["w"] = w
        st["ws"] = torch.rand(N, device="cuda", generator=g).mul_(2e-3).add_(1e-4)
        dt = _DT[case["out"]]
        st["bias"] = _normal(g, N).to(dt) if case["bias"] else None
        st["out"] = torch.empty(T, N, dtype=dt, device="cuda")
    else:
        V, dt = case["V"], _DT[case["dtype"]]
        x = torch.empty(T, V, dtype=dt, device="cuda")
        for i in range(0, T, 256):
            n = min(256, T - i)
            c = _normal(g, n, V).mul_(2.5)
            # the context's likely tokens: forty places of their own in each row
            at = torch.randint(V, (n, 1), device="cuda", generator=g) + torch.arange(40, device="cuda") * (V // 41)
            c.scatter_(1, at % V, 6.0 + 4.0 * _normal(g, n, 40))
            if case["masked"]:
                c[torch.rand(V, device="cuda", generator=g).expand(n, V) < 0.6] = float("-inf")
            x[i:i + n] = c
        ids = torch.randint(V, (T,), device="cuda", generator=g, dtype=torch.int32)
        best = x.argmax(1).to(torch.int32)  # most given tokens are the likeliest, the others are any
        st["ids"] = torch.where(torch.rand(T, device="cuda", generator=g) < 0.6, best, ids)
        st["x"] = x
        i32 = dict(dtype=torch.int32, device="cuda")
        st["out"] = (torch.empty(T, **f32), torch.empty(T, **i32), torch.empty(T, **f32),
                     torch.empty(T, case["top"], **i32), torch.empty(T, case["top"], **f32))
    return st


def run(st):
    c = st["case"]
    f = _own if own else _plain
    return f(c, st)


def _own(c, st):
    import any_precision_weight_gb300 as pw
    op = c["op"]
    if op == "norm":
        if not c["i8"]:
            y = pw.pw_rms_norm(st["x"], st["w"], EPS, residual=st["res"], out=st["y"], sum_out=st["sum"])
            return {"y": y[0], "sum": y[1]} if c["residual"] else {"y": y}
        r = pw.pw_rms_norm_i8(st["x"], st["w"], EPS, residual=st["res"], q=st["q"], scale=st["scale"],
                              sum_out=st["sum"])
        out = {"y": torch.mul(r[0], r[1].unsqueeze(1), out=st["y"]), "scale": r[1]}
        if c["residual"]:
            out["sum"] = r[2]
        return out
    if op == "quant":
        q, s = pw.pw_quant_i8(st["x"], q=st["q"], scale=st["scale"])
        return {"y": torch.mul(q, s.unsqueeze(1), out=st["y"]), "scale": s}
    if op == "linear":
        return {"out": pw.pw_linear_i8(st["x"], st["xs"], st["w"], st["ws"], bias=st["bias"], out=st["out"])}
    r = pw.pw_logprobs(st["x"], st["ids"], top=c["top"], out=st["out"])
    return _named(r, c["top"])


def _named(r, top):
    out = {"logprob": r[0], "rank": r[1], "entropy": r[2]}
    if top:
        out["top_ids"], out["top_logprobs"] = r[3], r[4]
    return out


def _quantised(y):
    """(values that the int8 rows stand for, scales) of 32-bit rows."""
    scale = y.abs().amax(1, keepdim=True) / 127
    q = torch.where(scale > 0, (y / scale).round(), torch.zeros_like(y))
    return q * scale, scale.squeeze(1)


def _plain(c, st):
    op = c["op"]
    if op == "norm":
        s = st["x"].float()
        out = {}
        if c["residual"]:
            s = s + st["res"].float()
            out["sum"] = s.to(st["x"].dtype)
        y = s * torch.rsqrt(s.square().mean(1, keepdim=True) + EPS) * st["w"].float()
        if c["i8"]:
            y, out["scale"] = _quantised(y)
        out["y"] = y.to(st["x"].dtype)
        return out
    if op == "quant":
        y, scale = _quantised(st["x"].float())
        return {"y": y.to(st["y"].dtype), "scale": scale}
    if op == "linear":
        a = st["x"].float() @ st["w"].float().t()
        a = a * st["xs"].unsqueeze(1) * st["ws"]
        if st["bias"] is not None:
            a = a + st["bias"].float()
        return {"out": a.to(st["out"].dtype)}
    x = st["x"].float()
    V = x.shape[1]
    m = x.amax(1, keepdim=True)
    e = (x - m).exp()
    s = e.sum(1, keepdim=True)
    lse = m + s.log()
    u = torch.where(e > 0, (x - m) * e, torch.zeros_like(e)).sum(1, keepdim=True)
    ids = st["ids"].long().unsqueeze(1)
    xt = x.gather(1, ids)
    before = torch.arange(V, device=x.device) < ids
    rank = ((x > xt) | ((x == xt) & before)).sum(1, dtype=torch.int32)
    out = {"logprob": (xt - lse).squeeze(1), "rank": rank, "entropy": (s.log() - u / s).squeeze(1)}
    if c["top"]:
        v, i = torch.sort(x, dim=1, descending=True, stable=True)  # ties: lowest index first
        out["top_ids"] = i[:, :c["top"]].to(torch.int32)
        out["top_logprobs"] = v[:, :c["top"]] - lse
    return out


def work(case):
    op, T = case["op"], case["T"]
    if op == "norm":
        n = T * case["H"]
        b = 2 * n * (3 if case["residual"] else 1) + 2 * case["H"]  # x, residual, sum; weight
        b += n + 4 * T if case["i8"] else 2 * n
        return {"bytes": b, "flops": 6 * n}
    if op == "quant":
        n = T * case["K"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + n + 4 * T, "flops": 3 * n}
    if op == "linear":
        N, K = case["N"], case["K"]
        o = 4 if case["out"] == "f32" else 2
        return {"bytes": N * K + T * K + 4 * (N + T) + T * N * o + (N * o if case["bias"] else 0),
                "flops": 2 * T * N * K}
    n = T * case["V"]
    return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + T * (16 + 8 * case["top"]), "flops": 6 * n}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]

    def quantised(y):
        a = y.abs().max(dim=1).values / 127
        q = torch.round(y / a[:, None].clamp(min=1e-300))
        return q * a[:, None], a

    if op == "norm":
        s = st["x"].double()
        out = {}
        if case["residual"]:
            s = s + st["res"].double()
            out["sum"] = s
        out["y"] = s / torch.sqrt((s * s).mean(dim=1)[:, None] + EPS) * st["w"].double()
        if case["i8"]:
            out["y"], out["scale"] = quantised(out["y"])
        return out
    if op == "quant":
        y, a = quantised(st["x"].double())
        return {"y": y, "scale": a}
    if op == "linear":
        x, xs, ws = st["x"].double(), st["xs"].double(), st["ws"].double()
        o = torch.empty(x.shape[0], st["w"].shape[0], dtype=torch.float64, device=x.device)
        for i in range(0, st["w"].shape[0], 16384):  # whole numbers: exact in 64-bit sums
            o[:, i:i + 16384] = (x @ st["w"][i:i + 16384].double().t()) * (xs[:, None] * ws[i:i + 16384])
        if st["bias"] is not None:
            o += st["bias"].double()
        return {"out": o}
    T, k = st["x"].shape[0], case["top"]
    lp = torch.empty(T, dtype=torch.float64, device="cuda")
    ent, top = torch.empty_like(lp), torch.empty(T, k, dtype=torch.float64, device="cuda")
    for i in range(0, T, 64):
        x = st["x"][i:i + 64].double()
        l = x - torch.logsumexp(x, dim=1, keepdim=True)
        p = torch.exp(l)
        ent[i:i + 64] = -(p * l).nan_to_num(0.0).sum(dim=1)
        lp[i:i + 64] = l.gather(1, st["ids"][i:i + 64].long()[:, None])[:, 0]
        if k:
            top[i:i + 64] = torch.topk(l, k, dim=1).values
    out = {"logprob": lp, "rank": None, "entropy": ent}
    if k:
        out["top_ids"], out["top_logprobs"] = None, top
    return out
