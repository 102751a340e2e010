"""Cases of the operators of an expert layer in 8-bit floating point, for timing
and comparison.

Each case is one call of one operator on seeded inputs: the quantisers to e4m3
with a scale for every 128 columns (pw_quant_f8, pw_silu_quant_f8,
pw_quant_f8_blocks), the product of such rows with weights that have a scale for
each 128 x 128 block (pw_linear_f8), the same for rows sorted by expert
(pw_grouped_linear_f8), the routing (pw_route) and the experts' weighted sum
(pw_combine).  ``run`` computes it in plain torch operations in 32 bits, or, where
``own`` is true, by the framework's entry points; ``exact`` restates it in 64 bits.
"""
from __future__ import annotations

import numpy as np
import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
TOP = 448.0   # largest e4m3 number
B = 128       # columns, and rows of weights, that share a scale


def listed():
    return [
        # a decode batch of 4 tokens, each for its 4 experts of 60: rows gathered in expert order
        dict(name="quant_step", op="quant", form="rows", T=16, K=2048, dtype="f16", per=4),
        # a prompt of 2048 tokens for 2 experts each: SiLU(gate) * up between the two expert products
        dict(name="quant_act_prefill", op="quant", form="act", T=4096, K=14336, dtype="f16", per=1),
        # one sequence's decode step through a wide projection: weights stream once
        dict(name="linear_step", op="linear", T=1, N=28672, K=4096, out="f16", bias=False),
        # ragged batch and odd sizes, with a bias
        dict(name="linear_ragged", op="linear", T=201, N=2891, K=1411, out="bf16", bias=True),
        # a prompt batch through a wide projection: tensor bound
        dict(name="linear_prefill", op="linear", T=2048, N=28672, K=4096, out="f16", bias=False),
        # a decode batch of 4 tokens in 2 of 8 wide experts: the weights of those that were chosen stream once
        dict(name="grouped_step", op="grouped", R=8, E=8, N=28672, K=4096, out="f16", bias=False),
        # a decode batch of 64 tokens in 4 of 60 narrow experts: a few rows to each
        dict(name="grouped_decode", op="grouped", R=256, E=60, N=2048, K=1408, out="f32", bias=False),
        # a prompt of 2048 tokens in 2 of 8 wide experts: ragged groups of hundreds of rows, tensor bound
        dict(name="grouped_prefill", op="grouped", R=4096, E=8, N=28672, K=4096, out="f16", bias=False),
        # the routing of a decode batch of 4: latency only
        dict(name="route_step", op="route", T=4, E=60, k=4, renorm=False),
        # the routing of a long prompt batch
        dict(name="route_prefill", op="route", T=8192, E=60, k=4, renorm=True),
        # the experts' sum of one sequence's decode step: latency only
        dict(name="combine_step", op="combine", T=1, H=4096, k=2, y="f16", out="f16", residual=True),
        # the experts' sum of a prompt batch on top of a shared expert's output
        dict(name="combine_prefill", op="combine", T=8192, H=4096, k=2, y="f16", out="f16", residual=True),
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
    op = rng.choice(["quant", "linear", "linear", "grouped", "grouped", "route", "combine"])
    if op == "quant":
        form = rng.choice(["rows", "act", "blocks"])
        K = _log(rng, 64, 14336)
        T = _log(rng, 1, max(1, min(8192, 4096 * 14336 // K)))
        return dict(op=op, form=form, T=T, K=K, dtype=rng.choice(["f16", "bf16", "f32"]),
                    per=rng.choice([1, 2, 4]) if form == "rows" else 1)
    if op == "linear":
        K = _log(rng, 64, 14336)
        N = _log(rng, 8, min(131072, 131072 * 4096 // K))
        T = _log(rng, 1, max(1, min(4096, 2048 * 28672 * 4096 // (N * K), (1 << 28) // N)))
        return dict(op=op, T=T, N=N, K=K, out=rng.choice(["f16", "bf16", "f32"]), bias=rng.random() < 0.3)
    if op == "grouped":
        E = _log(rng, 2, 128)
        K = _log(rng, 64, 14336)
        N = _log(rng, 64, max(64, min(28672, 8 * 28672 * 4096 // (E * K))))
        R = _log(rng, 1, max(1, min(8192, 4096 * 28672 * 4096 // (N * K), (1 << 28) // N)))
        return dict(op=op, R=R, E=E, N=N, K=K, out=rng.choice(["f16", "bf16", "f32"]), bias=rng.random() < 0.2)
    if op == "route":
        E = _log(rng, 2, 256)
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E)), renorm=rng.random() < 0.5)
    H, k = _log(rng, 64, 14336), rng.randint(1, 8)
    T = _log(rng, 1, max(1, min(8192, 8192 * 4096 * 2 // (H * k))))
    return dict(op=op, T=T, H=H, k=k, y=rng.choice(["f16", "bf16", "f32"]), out=rng.choice(["f16", "bf16", "f32"]),
                residual=rng.random() < 0.6)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _blocks(n):
    return (n + B - 1) // B


def _rows_f8(*shape):
    """e4m3 rows that start on 16-byte boundaries, as the quantisers lay them out."""
    return torch.empty(*shape[:-1], (shape[-1] + 15) // 16 * 16, dtype=F8, device="cuda")[..., :shape[-1]]


def _activations(g, T, K):
    """Hidden states as models have them: normal, a hundredth of the channels much larger."""
    x = _normal(g, T, K)
    big = 1.0 + 15.0 * (torch.rand(K, device="cuda", generator=g) < 0.01)
    return x.mul_(big)


def _spread(s, rows, K):
    """Scales of blocks at every element of [..][K]; rows: how many rows share one (or 1)."""
    s = s.repeat_interleave(B, -1)[..., :K]
    return s if rows == 1 else s.repeat_interleave(rows, -2)


def _quantised(x, scale, rows):
    """e4m3 rows of x for given scales: inputs that are 8-bit from the start."""
    q = _rows_f8(*x.shape)
    K = x.shape[-1]
    q.copy_((x / _spread(scale, rows, K)[..., :x.shape[-2], :]).clamp_(-TOP, TOP).to(F8))
    return q


def _row_values(x):
    T, K = x.shape
    p = torch.nn.functional.pad(x, (0, _blocks(K) * B - K)).view(T, -1, B)
    s = (p.abs().amax(2) / TOP).clamp_(min=1e-12)
    return _quantised(x, s, 1), s


def _weight_values(g, N, K):
    """Weights of a checkpoint: normal rows, each 128 x 128 block a size of its own."""
    w = _normal(g, N, K).mul_(K ** -0.5)
    s = torch.rand(_blocks(N), _blocks(K), device="cuda", generator=g).add_(0.5).mul_(4.5 * K ** -0.5 / TOP)
    return _quantised(w, s, B), s


def _counts(case, seed):
    """Rows of each group: shares that differ as a router's do."""
    rng = np.random.default_rng(seed)
    return rng.multinomial(case["R"], rng.dirichlet(np.ones(case["E"])))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    f32 = dict(dtype=torch.float32, device="cuda")
    if op == "quant":
        T, K, dt = case["T"], case["K"], _DT[case["dtype"]]
        if case["form"] == "rows":
            n = -(-T // case["per"])
            st["x"] = _activations(g, n, K).to(dt)
            # the order that a routing gives: pair ids, `per` to a token
            st["rows"] = torch.randperm(n * case["per"], device="cuda", generator=g)[:T].to(torch.int32)
        elif case["form"] == "act":
            st["x"] = _normal(g, T, 2 * K).mul_(1.5).to(dt)
        else:
            st["x"] = _normal(g, T, K).mul_(K ** -0.5).to(dt)
        st["q"] = _rows_f8(T, K)
        st["scale"] = torch.empty(_blocks(T) if case["form"] == "blocks" else T, _blocks(K), **f32)
    elif op == "linear":
        T, N, K, dt = case["T"], case["N"], case["K"], _DT[case["out"]]
        st["x"], st["xs"] = _row_values(_activations(g, T, K))
        st["w"], st["ws"] = _weight_values(g, N, K)
        st["bias"] = _normal(g, N).to(dt) if case["bias"] else None
        st["out"] = torch.empty(T, N, dtype=dt, device="cuda")
    elif op == "grouped":
        R, E, N, K, dt = case["R"], case["E"], case["N"], case["K"], _DT[case["out"]]
        counts = _counts(case, seed)
        st["counts"], st["most"] = [int(c) for c in counts], int(counts.max())
        st["offsets"] = torch.from_numpy(np.concatenate([[0], counts.cumsum()]).astype(np.int32)).cuda()
        st["x"], st["xs"] = _row_values(_activations(g, R, K))
        st["w"], st["ws"] = _rows_f8(E, N, K), torch.empty(E, _blocks(N), _blocks(K), **f32)
        for e in range(E):
            w, s = _weight_values(g, N, K)
            st["w"][e].copy_(w)
            st["ws"][e].copy_(s)
        st["bias"] = _normal(g, E, N).to(dt) if case["bias"] else None
        st["out"] = torch.empty(R, N, dtype=dt, device="cuda")
    elif op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # logits of a 16-bit router: equal ones now and then; experts of uneven popularity
        st["x"] = (_normal(g, T, E) + _normal(g, E)).to(torch.bfloat16).float()
        i32 = dict(dtype=torch.int32, device="cuda")
        st["out"] = (torch.empty(T, k, **i32), torch.empty(T, k, **f32), torch.empty(E + 1, **i32),
                     torch.empty(T * k, **i32), torch.empty(T * k, **i32))
    else:
        T, H, k = case["T"], case["H"], case["k"]
        st["y"] = _normal(g, T * k, H).to(_DT[case["y"]])
        st["w"] = torch.rand(T, k, device="cuda", generator=g)
        st["w"] /= st["w"].sum(1, keepdim=True)
        st["inv"] = torch.randperm(T * k, device="cuda", generator=g).to(torch.int32)
        dt = _DT[case["out"]]
        st["res"] = _normal(g, T, H).mul_(2).to(dt) if case["residual"] else None
        st["out"] = torch.empty(T, H, dtype=dt, device="cuda")
    return st


def run(st):
    c = st["case"]
    f = _own if own else _plain
    return f(c, st)


def _own(c, st):
    import any_precision_weight_gb300 as pw
    op = c["op"]
    if op == "quant":
        if c["form"] == "rows":
            r = pw.pw_quant_f8(st["x"], rows=st["rows"], per=c["per"], q=st["q"], scale=st["scale"])
        elif c["form"] == "act":
            r = pw.pw_silu_quant_f8(st["x"], q=st["q"], scale=st["scale"])
        else:
            r = pw.pw_quant_f8_blocks(st["x"], q=st["q"], scale=st["scale"])
        return {"q": r[0], "scale": r[1]}
    if op == "linear":
        return {"out": pw.pw_linear_f8(st["x"], st["xs"], st["w"], st["ws"], bias=st["bias"], out=st["out"])}
    if op == "grouped":
        return {"out": pw.pw_grouped_linear_f8(st["x"], st["xs"], st["w"], st["ws"], st["offsets"], bias=st["bias"],
                                               out=st["out"])}
    if op == "route":
        return dict(pw.pw_route(st["x"], c["k"], c["renorm"], out=st["out"])._asdict())
    return {"out": pw.pw_combine(st["y"], st["w"], st["inv"], residual=st["res"], out=st["out"])}


def _plain_quant(c, st):
    x = st["x"].float()
    if c["form"] == "rows":
        x = x[torch.div(st["rows"], c["per"], rounding_mode="floor").long()]
    elif c["form"] == "act":
        gate, up = x.chunk(2, dim=1)
        x = gate / (1 + (-gate).exp()) * up
    T, K = x.shape
    rows = B if c["form"] == "blocks" else 1
    nb = -(-T // rows)
    p = torch.nn.functional.pad(x, (0, _blocks(K) * B - K, 0, nb * rows - T)).view(nb, rows, -1, B)
    top = p.abs().amax((1, 3), keepdim=True)
    # in 64 bits: quotients next to a border of e4m3
    v = torch.where(top > 0, p.double() * TOP / top.double(), torch.zeros_like(p, dtype=torch.float64))
    q = v.float().to(F8).view(nb * rows, -1)[:T, :K]
    return {"q": q, "scale": (top / TOP).view(nb, -1)}


def _plain(c, st):
    op = c["op"]
    if op == "quant":
        return _plain_quant(c, st)
    if op in ("linear", "grouped"):
        K, N = c["K"], c["N"]
        x = st["x"].float() * _spread(st["xs"], 1, K)
        w = st["w"].float() * _spread(st["ws"], B, K)[..., :N, :]
        if op == "linear":
            a = x @ w.t()
            if st["bias"] is not None:
                a = a + st["bias"].float()
            return {"out": a.to(st["out"].dtype)}
        off, r = st["offsets"].long(), torch.arange(c["R"], device=x.device)
        e = (r.unsqueeze(1) >= off[1:]).sum(1)
        at = r - off[e]
        padded = torch.zeros(c["E"], st["most"], K, device=x.device)
        padded[e, at] = x
        a = torch.bmm(padded, w.transpose(1, 2))[e, at]
        if st["bias"] is not None:
            a = a + st["bias"].float()[e]
        return {"out": a.to(st["out"].dtype)}
    if op == "route":
        x, k = st["x"], c["k"]
        v, i = torch.sort(x, dim=1, descending=True, stable=True)   # ties: lowest index first
        p = (v - v[:, :1]).exp()
        w = p[:, :k] / (p[:, :k].sum(1, keepdim=True) if c["renorm"] else p.sum(1, keepdim=True))
        idx = i[:, :k]
        flat = idx.reshape(-1)
        perm = torch.sort(flat, stable=True).indices
        inv = torch.empty_like(perm)
        inv[perm] = torch.arange(flat.numel(), device=x.device)
        counts = (flat.unsqueeze(1) == torch.arange(c["E"], device=x.device)).sum(0)
        off = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
        i32 = torch.int32
        return {"idx": idx.to(i32), "weight": w, "offsets": off.to(i32), "perm": perm.to(i32), "inv": inv.to(i32)}
    T, k = c["T"], c["k"]
    a = (st["y"].float()[st["inv"].long()].view(T, k, -1) * st["w"].unsqueeze(2)).sum(1)
    if st["res"] is not None:
        a = a + st["res"].float()
    return {"out": a.to(st["out"].dtype)}


def work(case):
    op = case["op"]
    size = lambda d: 4 if d == "f32" else 2
    if op == "quant":
        T, K, s = case["T"], case["K"], size(case["dtype"])
        n = -(-T // case["per"]) * K * (2 if case["form"] == "act" else 1)
        scales = (_blocks(T) if case["form"] == "blocks" else T) * _blocks(K)
        return {"bytes": n * s + T * K + 4 * scales + (4 * T if case["form"] == "rows" else 0),
                "flops": T * K * (8 if case["form"] == "act" else 3)}
    if op == "linear":
        T, N, K, o = case["T"], case["N"], case["K"], size(case["out"])
        return {"bytes": N * K + T * K + 4 * (T + _blocks(N)) * _blocks(K) + T * N * o + (N * o if case["bias"] else 0),
                "flops": 2 * T * N * K}
    if op == "grouped":
        R, E, N, K, o = case["R"], case["E"], case["N"], case["K"], size(case["out"])
        # groups that R rows reach when each expert's share is uniform over the simplex
        busy = E * R / (E + R - 1)
        return {"bytes": busy * (N * K + 4 * _blocks(N) * _blocks(K) + (N * o if case["bias"] else 0)) + R * K
                + 4 * R * _blocks(K) + R * N * o + 4 * (E + 1), "flops": 2 * R * N * K}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + 16 * T * k + 4 * (E + 1), "flops": 4 * T * E}
    T, H, k, o = case["T"], case["H"], case["k"], size(case["out"])
    return {"bytes": T * k * (H * size(case["y"]) + 8) + T * H * o * (2 if case["residual"] else 1),
            "flops": 2 * T * k * H}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        # the quotients before their rounding to 8 bits, which is the output's type
        x = st["x"].double()
        if case["form"] == "rows":
            x = x[(st["rows"].long() // case["per"])]
        elif case["form"] == "act":
            K = case["K"]
            x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
        T, K = x.shape
        step = B if case["form"] == "blocks" else 1
        scale = torch.zeros(-(-T // step), _blocks(K), dtype=torch.float64, device=x.device)
        for b in range(_blocks(K)):
            part = x[:, b * B:(b + 1) * B]
            m = part.abs().amax(1)
            if step > 1:
                m = torch.stack([m[i:i + step].max() for i in range(0, T, step)])
            scale[:, b] = m / TOP
            s = m.repeat_interleave(step)[:T, None]
            part.mul_(TOP).div_(torch.where(s > 0, s, torch.ones_like(s)))
        return {"q": x, "scale": scale}
    if op in ("linear", "grouped"):
        K, N = case["K"], case["N"]
        cols = torch.arange(K, device="cuda") // B
        x = st["x"].double() * st["xs"].double()[:, cols]
        out = torch.zeros(x.shape[0], N, dtype=torch.float64, device="cuda")
        groups = [(0, x.shape[0], st["w"], st["ws"], st["bias"])]
        if op == "grouped":
            ends = np.cumsum(st["counts"])
            groups = [(int(z) - n, int(z), st["w"][e], st["ws"][e], None if st["bias"] is None else st["bias"][e])
                      for e, (n, z) in enumerate(zip(st["counts"], ends))]
        for a, z, w, ws, bias in groups:
            if z == a:
                continue
            for n in range(0, N, 8192):
                m = min(N, n + 8192)
                rows = torch.arange(n, m, device="cuda") // B
                out[a:z, n:m] = x[a:z] @ (w[n:m].double() * ws.double()[rows][:, cols]).t()
            if bias is not None:
                out[a:z] += bias.double()
        return {"out": out}
    if op == "route":
        x, k = st["x"].double(), case["k"]
        top = torch.topk(x, k, dim=1).values
        w = torch.exp(top - (torch.logsumexp(top if case["renorm"] else x, dim=1)[:, None]))
        return {"idx": None, "weight": w, "offsets": None, "perm": None, "inv": None}
    out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
    inv = st["inv"].view(case["T"], case["k"]).long()
    for j in range(case["k"]):
        out += st["w"][:, j:j + 1].double() * st["y"][inv[:, j]].double()
    if st["res"] is not None:
        out += st["res"].double()
    return {"out": out}
