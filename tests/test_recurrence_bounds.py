"""The bounds of recurrence_bounds.py on the CPU: the formulas in fp32 keep them, and losses of precision that a kernel could have
do not."""
import functools

import pytest
import torch

import layer_ref as ref
from recurrence_bounds import Bounds

B, L, D = 2, 600, 24


def bf16(t):
    return t.bfloat16().float()


def inputs(slow):
    g = torch.Generator().manual_seed(11 + slow)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    A = torch.log(0.9 + 0.099 * torch.rand(D, generator=g)) if slow else -torch.exp(rn(D) - 2).clamp(max=2.0)
    return rn(B, L, D), 2 * rn(B, L, D), A, 2 * rn(B, L, D), rn(D), rn(D), rn(B, D), rn(B, L, D), rn(B, D)


def in_fp32(x, gate, A, ig, gb, ib, h0, dout, dfin, fault=None):
    """Outputs and gradients token by token in fp32, one thing less precise by ``fault``."""
    r, i = torch.sigmoid(gate + gb), torch.sigmoid(ig + ib)
    rc, ic = torch.sigmoid(-(gate + gb)), torch.sigmoid(-(ig + ib))  # (1 - r loses an open gate's)
    if fault == "gate":
        r = bf16(r)
    low = A * r
    a = torch.exp(low)
    if fault == "decay":
        a = torch.exp(low.half().float())
    beta = torch.sqrt(1 - a * a if fault == "beta" else -torch.expm1(2 * low))
    if fault == "root":
        beta = beta * (1 + 2.0**-12)
    added = beta * i * x
    h, hs, before = h0, [], []
    for t in range(L):
        if t % 128 == 0 and t and fault == "state":
            h = bf16(h)
        before.append(h)
        h = a[:, t] * h + added[:, t]
        hs.append(h)
    v, dx, dgate, dA, dig = dfin, [], [], [], []
    for t in reversed(range(L)):
        if t % 64 == 63 and t != L - 1 and fault == "gradient":
            v = bf16(v)
        g = dout[:, t] + v
        hb = bf16(before[t]) if fault == "kept" else before[t]
        dl = a[:, t] * g * (hb - a[:, t] * i[:, t] * x[:, t] / beta[:, t])
        dx.append(g * beta[:, t] * i[:, t])
        dig.append(g * added[:, t] * ic[:, t])
        dgate.append(dl * A * r[:, t] * rc[:, t])
        dA.append(dl * r[:, t])
        v = a[:, t] * g
    dx, dgate, dA, dig = (torch.stack(z[::-1], 1) for z in (dx, dgate, dA, dig))
    over = lambda z: z.sum((0, 1))  # noqa: E731
    return torch.stack(hs, 1), h, dx, dgate, over(dA), dig, over(dgate), over(dig), v


NAMES = ("out", "final state", "dx", "dgate", "dA", "din_gate", "dgate_bias", "din_bias", "dh0")


@functools.lru_cache(maxsize=None)
def expected(slow):
    *ins, h0, dout, dfin = inputs(slow)
    rr = [(b, b, 0, L) for b in range(B)]
    bound = Bounds(*ins, True, h0, B, rr, dout, dfin)
    out, fin, _ = ref.recurrence(*ins, True, h0, B, rr)
    return (out, fin) + ref.recurrence_grads(dout, dfin, *ins, True, h0, B, rr), (bound.out, bound.fin) + bound.grads


def check(slow, fault):
    """Names of the outputs that pass their bounds."""
    passed = set()
    for v, w, e, name in zip(in_fp32(*inputs(slow), fault), *expected(slow), NAMES):
        try:
            ref.close(v, w, e, 1, torch.float32, name)
            passed.add(name)
        except AssertionError:
            pass
    return passed


@pytest.mark.parametrize("slow", [False, True])
def test_fp32_keeps_the_bounds(slow):
    assert check(slow, None) == set(NAMES)


@pytest.mark.parametrize("slow", [False, True])
@pytest.mark.parametrize("fault,shows", [("state", {"out"}), ("gradient", {"dx", "dgate", "din_gate"}), ("kept", {"dgate"}),
                                         ("decay", {"out", "dx"}), ("gate", {"out", "dx"}), ("root", {"out", "dx"}),
                                         ("beta", {"out", "dx"})])
def test_lost_precision_is_seen(slow, fault, shows):
    assert not shows & check(slow, fault)
