"""64-bit references of the residual norm, the matrix product with its epilogue and the gated linear recurrence, from
their definitions.  The error bounds are those of selective_ref.py: with ``absolute=True`` a function gives its sums with
every product's absolute value, and a value with at most K roundings on the way from any input is within
K u of that."""
import math

import torch

from selective_ref import U, close, d64, runs  # noqa: F401


# ---- residual norm --------------------------------------------------------------------------------
def total(x, res):
    return d64(x) if res is None else d64(x) + d64(res)


def norm(x, res, w, eps):
    """(s, y)."""
    s = total(x, res)
    return s, s / (s.square().mean(-1, keepdim=True) + eps).sqrt() * d64(w)


def norm_grads(dout, s, w, dsum, eps, absolute=False):
    """(ds, dw): the formula's."""
    dout, s, w = d64(dout), d64(s), d64(w)
    r = 1 / (s.square().mean(-1, keepdim=True) + eps).sqrt()
    g, n = dout * w, s * r
    if absolute:
        g, n, dout = g.abs(), n.abs(), dout.abs()
    lead = tuple(range(s.dim() - 1))
    m = (g * n).mean(-1, keepdim=True)
    ds = r * (g + n * m if absolute else g - n * m)
    if dsum is not None:
        ds = ds + (d64(dsum).abs() if absolute else d64(dsum))
    return ds, (dout * n).sum(lead)


def code_step(q, fmt):
    """The distance of neighbouring codes at |q| (the larger one on a border)."""
    if fmt == "int8":
        return torch.ones_like(q)
    return torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)


# ---- matrix product -------------------------------------------------------------------------------
def act(v, kind):
    if kind == "silu":
        return v * torch.sigmoid(v)
    return 0.5 * v * (1 + torch.erf(v / math.sqrt(2))) if kind == "gelu" else v


def dact(v, kind):
    if kind == "silu":
        p = torch.sigmoid(v)
        return p * (1 + v * (1 - p))
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(v / math.sqrt(2))) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(v)


def product(x, w, bias=None, sx=None, sw=None, absolute=False):
    """pre [..., N]."""
    x, w, bias, sx, sw = d64(x.float()), d64(w.float()), d64(bias), d64(sx), d64(sw)
    if absolute:
        x, w, bias, sx, sw = (None if v is None else v.abs() for v in (x, w, bias, sx, sw))
    v = x @ w.t()
    v = v if sx is None else v * sx[..., None]
    v = v if sw is None else v * sw
    return v if bias is None else v + bias


def product_grads(dout, x, w, pre, kind, absolute=False):
    """(dx, dw, dbias): the formula's, and with ``absolute`` their sums of absolute values."""
    N, K = w.shape
    d = d64(dout).reshape(-1, N)
    if kind:
        d = d * dact(d64(pre).reshape(-1, N), kind)
    x, w = d64(x).reshape(-1, K), d64(w)
    if absolute:
        # act' is right to a few u of 1, so its part of the scale is at least that of 1
        d, x, w = d64(dout).reshape(-1, N).abs() * (1.2 if kind else 1), x.abs(), w.abs()
    return d @ w, d.t() @ x, d.sum(0)


# ---- gated recurrence -------------------------------------------------------------------------------
def gates(gate, A, ig, gb, ib, normalize):
    """(r, i, a, beta)."""
    gate, A, ig, gb, ib = d64(gate), d64(A), d64(ig), d64(gb), d64(ib)
    r = torch.sigmoid(gate if gb is None else gate + gb)
    i = torch.ones_like(r) if ig is None else torch.sigmoid(ig if ib is None else ig + ib)
    lo = A.clamp(min=-1e300) * r
    a = torch.exp(lo)
    return r, i, a, torch.sqrt(-torch.expm1(2 * lo)) if normalize else torch.ones_like(a)


def recurrence(x, gate, A, ig, gb, ib, normalize, h0, S, rr, absolute=False):
    """(h [B, L, D], final state [S, D], h before each token): loops over the tokens of every sequence of ``rr``."""
    x, h0 = d64(x), d64(h0)
    _, i, a, beta = gates(gate, A, ig, gb, ib, normalize)
    if absolute:
        x, h0 = x.abs(), None if h0 is None else h0.abs()
    out, before = torch.zeros_like(x), torch.zeros_like(x)
    fin = torch.zeros(S, x.shape[-1], dtype=torch.float64)
    for b, q, t0, n in rr:
        real = 0 <= q < S
        h = h0[q] if h0 is not None and real else torch.zeros(x.shape[-1], dtype=torch.float64)
        for t in range(t0, t0 + n):
            before[b, t] = h
            h = a[b, t] * h + beta[b, t] * i[b, t] * x[b, t]
            out[b, t] = h
        if real:
            fin[q] = h
    return out, fin, before


def recurrence_grads(dout, dfin, x, gate, A, ig, gb, ib, normalize, h0, S, rr, absolute=False):
    """(dx, dgate, dA, din_gate, dgate_bias, din_bias, dh0) by the formula; padding counts as nothing."""
    _, _, before = recurrence(x, gate, A, ig, gb, ib, normalize, h0, S, rr, absolute)
    r, i, a, beta = gates(gate, A, ig, gb, ib, normalize)
    x, dout, dfin, A = d64(x), d64(dout), d64(dfin), d64(A).clamp(min=-1e300)
    if absolute:
        x, dout, dfin, A = x.abs(), dout.abs(), None if dfin is None else dfin.abs(), A.abs()
    dx, dgate, dig, dA = (torch.zeros_like(x) for _ in range(4))
    dh0 = torch.zeros(S, x.shape[-1], dtype=torch.float64)
    for b, q, t0, n in rr:
        if not 0 <= q < S:
            continue
        v = dfin[q] if dfin is not None else torch.zeros(x.shape[-1], dtype=torch.float64)
        for t in reversed(range(t0, t0 + n)):
            g = dout[b, t] + v
            dl = a[b, t] * g * before[b, t]
            if normalize:
                root = torch.where(beta[b, t] > 0, a[b, t] ** 2 / beta[b, t].clamp(min=1e-300), 0) * g * i[b, t] * x[b, t]
                dl = dl + root if absolute else dl - root
            dx[b, t] = g * beta[b, t] * i[b, t]
            dgate[b, t] = dl * A * r[b, t] * (1 - r[b, t])
            dA[b, t] = dl * r[b, t]
            dig[b, t] = g * beta[b, t] * x[b, t] * i[b, t] * (1 - i[b, t])
            v = a[b, t] * g
        dh0[q] = v
    over = lambda t: t.sum((0, 1))  # noqa: E731
    return dx, dgate, over(dA), dig, over(dgate), over(dig), dh0
