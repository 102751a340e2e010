"""The barriers between the roles of pw_linear_i8's tensor-core kernels, modelled on
the host: no warp may pass a wait before the load or the product that it waits for.

The converting groups take the stages in turn and wait by parity, and a parity
tells a use of a stage from the one before it only.  Loads have no order of
completion, so the model holds back each load in turn while every other warp
goes on as far as it can, and then lets loads land in random orders.  The ring
sizes are read from the kernels' source.
"""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "any_precision_weight_gb300",
                      "csrc", "pw_linear.cu")


def _value(text, name, env):
    """The value of `constexpr int NAME = ...;` (numbers, names, one a == b ? c : d)."""
    expr = re.search(r"constexpr (?:int|bool) (?:\w+ = [^;]*, )?%s = ([^;,]+)[;,]" % name, text).group(1)
    expr = re.sub(r"^(.*?)\?(.*):(.*)$", r"((\2) if (\1) else (\3))", expr.strip())
    return eval(expr.replace("/", "//"), {}, env)


def _rings(name):
    """(converting groups, warps of one, operand stages S, int8 stages S8, whether a
    group waits for its operand stage before the weights) of a kernel."""
    text = open(SOURCE).read()
    env = {"kConvWarps": _value(text, "kConvWarps", {})}
    cls, _, mt = name.partition(" ")
    body = re.search(r"struct %s \{\n(.*?)\n\};" % cls, text, re.S).group(1)
    if mt:
        env["MT"] = int(mt)
    groups = body if "kGroups =" in body else text
    env["kGroups"] = _value(groups, "kGroups", env)
    first = "kOperandFirst" in body and _value(body, "kOperandFirst", env)
    return env["kGroups"], _value(groups, "kGroupWarps", env), _value(body, "S", env), _value(body, "S8", env), first


class Barrier:
    def __init__(self, count):
        self.count, self.arrived, self.phase = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phase = 0, self.phase + 1

    def passed(self, parity):
        """What a parity wait asks: has the phase of this parity, the current one or the one before, ended."""
        return (self.phase - 1) & 1 == parity


class Early(Exception):
    pass


def _run(groups, warps, S, S8, operand_first, steps, held, rng=None):
    """One run of a CTA's roles over `steps` stages.  `held`: the load that lands only when
    nothing else can move (without rng).  Raises Early where a warp goes ahead of its stage."""
    full8, empty8 = [Barrier(1) for _ in range(S8)], [Barrier(warps) for _ in range(S8)]
    fullw, empty = [Barrier(warps) for _ in range(S)], [Barrier(1) for _ in range(S)]
    flying, holds = [], [None] * S8     # loads under way; the step whose bytes a stage holds
    done = [0]                          # products so far

    def loader():
        for k in range(steps):
            i, lap = k % S8, k // S8
            while lap and not empty8[i].passed((lap & 1) ^ 1):
                yield False
            flying.append(k)
            yield True

    def converter(group):
        for k in range(group, steps, groups):
            i8, i = k % S8, k % S
            while operand_first and k >= S and not empty[i].passed(((k // S) & 1) ^ 1):
                yield False
            while not full8[i8].passed((k // S8) & 1):
                yield False
            if holds[i8] != k:
                raise Early(f"step {k} is converted while the stage holds {holds[i8]}")
            while k >= S and not empty[i].passed(((k // S) & 1) ^ 1):
                yield False
            if done[0] < k - S + 1:
                raise Early(f"step {k} overwrites the operands of step {k - S}")
            fullw[i].arrive()
            empty8[i8].arrive()
            yield True

    def products():
        for k in range(steps):
            while not fullw[k % S].passed((k // S) & 1):
                yield False
            done[0] = k + 1
            empty[k % S].arrive()
            yield True

    roles = [loader(), products()] + [converter(g) for g in range(groups) for _ in range(warps)]
    live = set(range(len(roles)))

    def land(k):
        flying.remove(k)
        holds[k % S8] = k
        full8[k % S8].arrive()

    while live or flying:
        moved = False
        order = sorted(live)
        if rng:
            rng.shuffle(order)
        for r in order:
            try:
                moved |= next(roles[r])
            except StopIteration:
                live.discard(r)
                moved = True
        ready = [k for k in flying if rng or k != held]
        if rng and ready and (not moved or rng.random() < 0.5):
            land(rng.choice(ready))
            moved = True
        elif not rng and ready:
            land(ready[0])
            moved = True
        if not moved:
            if not flying:
                raise Early("the roles wait for one another")
            land(flying[0])
    if done[0] != steps:
        raise Early(f"{done[0]} products of {steps}")


def _all_orders(groups, warps, S, S8, operand_first=False):
    steps = 4 * S8 + 3
    for held in range(steps):
        _run(groups, warps, S, S8, operand_first, steps, held)
    for seed in range(200):
        _run(groups, warps, S, S8, operand_first, steps, None, random.Random(seed))


@pytest.mark.parametrize("kernel", ["Tile", "Thin 32", "Thin 64", "Thin 128"])
def test_no_wait_passes_a_lap_early(kernel):
    _all_orders(*_rings(kernel))


@pytest.mark.parametrize("groups,S,S8", [(4, 5, 7), (2, 4, 5), (2, 3, 3)])
def test_the_model_finds_rings_that_let_a_group_run_ahead(groups, S, S8):
    """Neither another group's load nor a product orders step s - S8 before step s here."""
    with pytest.raises(Early):
        _all_orders(groups, 2, S, S8)


@pytest.mark.parametrize("groups,S,S8", [(g, S, S8) for g in (1, 2, 4) for S in (3, 4, 5) for S8 in range(3, 11)
                                         if g <= S and g <= S8])
def test_the_condition_that_the_kernels_assert(groups, S, S8):
    """S8 a multiple of the groups (the group's own last load of the stage), or at least
    groups + S (a product that its own last stage waited for; S where the operand stage
    is waited for first): then no order goes wrong."""
    if S8 % groups == 0 or S8 >= groups + S:
        _all_orders(groups, 2, S, S8)
    if S8 % groups == 0 or S8 >= S:
        _all_orders(groups, 2, S, S8, True)
