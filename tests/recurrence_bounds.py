"""Bounds of the gated recurrence's outputs and gradients that go token by token, so that what a state forgets counts no more.

In units of u = 2^-24, for the formulas evaluated in fp32 with hops h -> p h + q joined in any order:
  exponent of a gate: t = -(v + bias) log2(e) in one fma, its constant and the scaled bias rounded before, so off by
      |t| + 1.45 |v| + 2.9 |bias|, which e = 2^t takes times ln 2, with 2 for the exponential
  gate s = 1 / (1 + e): (1 - s) of e's and 3 for the sum and the reciprocal; 1 - s = e s: e's and s's and 1
  decay a = exp(A r): |A r| times (r's and 3 roundings of the exponent), and 3
  beta = sqrt(1 - a^2): up to -2 A r = 1/2 by a polynomial of it, half of (r's and 5), and 2; from there by a, half of
      2 a^2 / (1 - a^2) times a's, and 2.5 (both are charged near the border)
  a term passing a token: a's own, the product's rounding, the sum's, and one for the joins of runs, waves and tiles (at most 10
      for 64 tokens); 20 once for a term's own sum and joins
so e[t] = a (e[t-1] + (a's + 3) H[t-1]) + (the addition's + 20) |added[t]|, H the states of absolute values, and likewise
backwards for the gradient.  Everything else is a product of values with such bounds.
"""
import torch

import layer_ref as ref
from selective_ref import d64


def gate_bound(v, bias, s):
    """(e's, s's, (1 - s)'s) in units of u."""
    b = torch.zeros_like(v) if bias is None else d64(bias).expand_as(v)
    e = 0.7 * (1.45 * (v + b).abs() + 1.45 * v.abs() + 2.9 * b.abs()) + 2
    one = (1 - s) * e + 3
    return e, one, e + one + 1


class Bounds:
    """Values and bounds (in units of u) of out, final state and, where dout is given, the gradients of ``sequences`` as
    layer_ref.recurrence and recurrence_grads take them."""

    def __init__(self, x, gate, A, ig, gb, ib, normalize, h0, S, sequences, dout=None, dfin=None):
        r, i, a, beta = ref.gates(gate, A, ig, gb, ib, normalize)
        x, h0, size = d64(x), d64(h0), d64(A).abs().clamp(max=1e300)
        _, er, ecr = gate_bound(d64(gate), gb, r)
        ei = eci = torch.zeros_like(r)
        if ig is not None:
            _, ei, eci = gate_bound(d64(ig), ib, i)
        low = size * r
        ea = low * (er + 3) + 3
        eb = torch.zeros_like(r)
        if normalize:
            past = a * a / (1 - a * a).clamp(min=1e-300) * ea + 2.5
            eb = (er + 5) / 2 + 2 + torch.where(2 * low > 0.45, past, torch.zeros_like(past))
        eu = ei + eb + 3
        added = (beta * i * x).abs()
        D = x.shape[-1]
        zero = torch.zeros(D, dtype=torch.float64)
        self.out, self.before, self.before_size = (torch.zeros_like(x) for _ in range(3))
        self.fin = torch.zeros(S, D, dtype=torch.float64)
        for b, q, t0, n in sequences:
            real = 0 <= q < S
            H = h0[q].abs() if h0 is not None and real else zero
            e = 20 * H
            for t in range(t0, t0 + n):
                self.before[b, t], self.before_size[b, t] = e, H
                e = a[b, t] * (e + (ea[b, t] + 3) * H) + (eu[b, t] + 20) * added[b, t]
                H = a[b, t] * H + added[b, t]
                self.out[b, t] = e
            if real:
                self.fin[q] = e
        if dout is None:
            return
        dout, dfin = d64(dout).abs(), None if dfin is None else d64(dfin).abs()
        parts = 30 + x.shape[0] * -(-x.shape[1] // 64)  # additions of a parameter's gradient: a tile's, and one a tile
        dx, dgate, dig, dA, sgate, sig, sA = (torch.zeros_like(x) for _ in range(7))
        dh0 = torch.zeros(S, D, dtype=torch.float64)
        for b, q, t0, n in sequences:
            if not 0 <= q < S:
                continue
            V = dfin[q] if dfin is not None else zero
            e = 20 * V
            for t in reversed(range(t0, t0 + n)):
                at, bt, it, rt, xt = a[b, t], beta[b, t], i[b, t], r[b, t], x[b, t].abs()
                G = dout[b, t] + V
                eg = e + 20 * dout[b, t] + G
                H, eh = self.before_size[b, t], self.before[b, t]
                dx[b, t] = bt * it * (eg + eu[b, t] * G)
                sig[b, t] = bt * it * (1 - it) * xt * G
                dig[b, t] = bt * it * (1 - it) * xt * (eg + (eu[b, t] + eci[b, t] + 4) * G)
                size_l = at * G * H
                dl = at * (eg * H + G * eh + (ea[b, t] + 4) * G * H)
                if normalize:
                    root = torch.where(bt > 0, at * at / bt.clamp(min=1e-300), 0) * it * xt
                    size_l = size_l + root * G
                    dl = dl + root * (eg + (2 * ea[b, t] + ei[b, t] + eb[b, t] + 8) * G)
                s = size * rt * (1 - rt)
                sgate[b, t] = s * size_l
                dgate[b, t] = s * (dl + (er[b, t] + ecr[b, t] + 6) * size_l)
                sA[b, t] = rt * size_l
                dA[b, t] = rt * (dl + (er[b, t] + 4) * size_l)
                e = at * (eg + (ea[b, t] + 3) * G)
                V = at * G
            dh0[q] = e
        over = lambda t, s: t.sum((0, 1)) + parts * s.sum((0, 1))  # noqa: E731
        self.grads = dx, dgate, over(dA, sA), dig, over(dgate, sgate), over(dig, sig), dh0
