"""64-bit references of the causal convolution, the selective scan and the 8-bit state cache, written as
loops over the definitions, and the error bounds that the GPU tests hold the kernels to.

Error bounds.  Every output is a sum of products of the inputs (and of exponentials, gates and
softplus values, each right to a few units in fp32).  A value computed in fp32 with at most K
roundings on the way from any input is within K u S of the exact one, u = 2^-24, where S is the same sum
with every product's absolute value; the last rounding to the output's type adds half a step, eps / 2
relative to the value.  S comes from the same loops with absolute values (``absolute=True``).
"""
import torch

U = 2.0 ** -24


def runs(B, L, seq_idx=None):
    """(batch row, state number, first token, tokens) of every sequence."""
    if seq_idx is None:
        return [(b, b, 0, L) for b in range(B)]
    out = []
    for b in range(B):
        t0 = 0
        for t in range(1, L + 1):
            if t == L or int(seq_idx[b, t]) != int(seq_idx[b, t0]):
                out.append((b, int(seq_idx[b, t0]), t0, t - t0))
                t0 = t
    return out


def d64(t):
    return None if t is None else t.detach().cpu().double()


def silu(v):
    return v * torch.sigmoid(v)


def dsilu(v):
    p = torch.sigmoid(v)
    return p * (1 + v * (1 - p))


def close(got, want, scale, roundings, dtype, name):
    """|got - want| <= eps/2 |want| + roundings u scale (plus the smallest steps of the type)."""
    got, want, scale = d64(got), d64(want), d64(scale)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fi = torch.finfo(dtype)
    # the last rounding is relative to the computed value, itself within the first term
    tol = (1 + fi.eps) * (fi.eps / 2 * want.abs() + roundings * U * scale) + fi.smallest_normal * fi.eps
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d values off, worst %.3g over its bound" % (
        name, int(bad.sum()), bad.numel(), float(((got - want).abs() / tol.clamp(min=1e-300))[bad].max()))


# ---- convolution ---------------------------------------------------------------------------------
def conv(x, w, bias, h0, S, act, rr, absolute=False):
    """(pre, out, final state [S, Ch, W-1], used): plain loops; ``absolute``: sums of absolute values (of pre)."""
    x, w, bias, h0 = d64(x), d64(w), d64(bias), d64(h0)
    Ch, W = w.shape
    if absolute:
        x, w, bias, h0 = (None if v is None else v.abs() for v in (x, w, bias, h0))
    pre = torch.zeros_like(x)
    fin = torch.zeros(S, Ch, W - 1, dtype=torch.float64)
    for b, q, t0, n in rr:
        old = h0[q].t() if h0 is not None and 0 <= q < S else torch.zeros(W - 1, Ch, dtype=torch.float64)
        line = torch.cat([old, x[b, t0:t0 + n]])
        for t in range(n):
            pre[b, t0 + t] = (line[t:t + W].t() * w).sum(1) + (0 if bias is None else bias)
        if 0 <= q < S:
            fin[q] = line[n:].t()
    return pre, (silu(pre) if act else pre), fin


def conv_grads(dout, dfin, x, w, bias, h0, S, act, rr, absolute=False):
    """dx, dw, dbias, dh0 by the definition's loops (or their absolute sums)."""
    pre, _, _ = conv(x, w, bias, h0, S, act, rr)
    x, w, h0, dout, dfin = d64(x), d64(w), d64(h0), d64(dout), d64(dfin)
    g = dout * (dsilu(pre) if act else 1)
    if absolute:
        # silu' is right to a few u of 1, so its part of the scale is at least that of 1
        g = dout.abs() * (1.1 if act else 1)
        x, w, h0, dfin = (None if v is None else v.abs() for v in (x, w, h0, dfin))
    Ch, W = w.shape
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), g.sum((0, 1))
    dh = torch.zeros(S, Ch, W - 1, dtype=torch.float64)
    for b, q, t0, n in rr:
        live = 0 <= q < S
        old = h0[q].t() if h0 is not None and live else torch.zeros(W - 1, Ch, dtype=torch.float64)
        line = torch.cat([old, x[b, t0:t0 + n]])
        dline = torch.zeros_like(line)
        for t in range(n):
            gt = g[b, t0 + t]
            dline[t:t + W] += (gt[:, None] * w).t()
            dw += gt[:, None] * line[t:t + W].t()
        if dfin is not None and live:
            dline[n:] += dfin[q].t()
        dx[b, t0:t0 + n] = dline[W - 1:]
        if live:
            dh[q] = dline[:W - 1].t()
    return dx, dw, db, dh


# ---- scan --------------------------------------------------------------------------------------------
def spread(v, Ch):
    return v.repeat_interleave(Ch // v.shape[-2], dim=-2)


def steps(dt, bias, softplus):
    v = d64(dt) + (0 if bias is None else d64(bias))
    return v, (torch.logaddexp(v, torch.zeros((), dtype=torch.float64)) if softplus else v)


def scan(x, dt, A, B, C, D, bias, z, h0, S, softplus, rr, absolute=False):
    """(out, final state [S, D, N], states after every token, y before the gate)."""
    x, A, B, C, D, z, h0 = (d64(t) for t in (x, A, B, C, D, z, h0))
    _, d = steps(dt, bias, softplus)
    if absolute:
        x, B, C, D, h0 = (None if t is None else t.abs() for t in (x, B, C, D, h0))
    dx = (d.abs() if absolute else d) * x
    Bt, L, Ch = x.shape
    N = A.shape[1]
    B, C = spread(B, Ch), spread(C, Ch)
    hs = torch.zeros(Bt, L, Ch, N, dtype=torch.float64)
    fin = torch.zeros(S, Ch, N, dtype=torch.float64)
    for b, q, t0, n in rr:
        live = 0 <= q < S
        h = h0[q] if h0 is not None and live else torch.zeros(Ch, N, dtype=torch.float64)
        for t in range(t0, t0 + n):
            h = torch.exp(d[b, t, :, None] * A) * h + dx[b, t, :, None] * B[b, t]
            hs[b, t] = h
        if live:
            fin[q] = h
    y = (hs * C).sum(-1) + (0 if D is None else D * x)
    gate = 1 if z is None else (silu(z).abs() if absolute else silu(z))
    return y * gate, fin, hs, y


def scan_grads(dout, dfin, x, dt, A, B, C, D, bias, z, h0, S, softplus, rr, absolute=False):
    """dict of dx, ddt, dA, dB, dC, dD, dbias, dz, dh0 (or their absolute sums)."""
    _, _, hs, y = scan(x, dt, A, B, C, D, bias, z, h0, S, softplus, rr, absolute)
    v, d = steps(dt, bias, softplus)
    x, A, B, C, D, z, h0, dout, dfin = (d64(t) for t in (x, A, B, C, D, z, h0, dout, dfin))
    decay = lambda b, t: torch.exp(d[b, t, :, None] * A)  # noqa: E731
    As, da, sz = A, d, None if z is None else silu(z)
    if absolute:
        x, B, C, D, h0, dout, dfin = (None if t is None else t.abs() for t in (x, B, C, D, h0, dout, dfin))
        As, da = A.abs(), d.abs()
        # the gate's own error is relative to its value, silu' is right to a few u of 1
        sz = None if z is None else sz.abs()
    Bt, L, Ch = x.shape
    G, N = B.shape[2:]
    Bc, Cc = spread(B, Ch), spread(C, Ch)
    dy = dout if z is None else dout * sz
    dz = None if z is None else dout * y * (1.1 if absolute else dsilu(z))
    dx, dd, dA, dh = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(A), torch.zeros(S, Ch, N, dtype=torch.float64)
    dB, dC = torch.zeros_like(B), torch.zeros_like(C)
    for b, q, t0, n in rr:
        live = 0 <= q < S
        g = dfin[q].clone() if dfin is not None and live else torch.zeros(Ch, N, dtype=torch.float64)
        for t in range(t0 + n - 1, t0 - 1, -1):
            prev = hs[b, t - 1] if t > t0 else (h0[q] if h0 is not None and live else torch.zeros(Ch, N, dtype=torch.float64))
            g = g + dy[b, t, :, None] * Cc[b, t]
            dC[b, t] = (dy[b, t, :, None] * hs[b, t]).view(G, -1, N).sum(1)
            dB[b, t] = (g * (da[b, t] * x[b, t])[:, None]).view(G, -1, N).sum(1)
            s = (g * Bc[b, t]).sum(-1)
            g = g * decay(b, t)
            qn = g * prev
            dA += da[b, t, :, None] * qn
            dd[b, t] = x[b, t] * s + (qn * As).sum(-1)
            dx[b, t] = da[b, t] * s + (0 if D is None else D * dy[b, t])
        if live:
            dh[q] = g
    ddt = dd * (torch.sigmoid(v) if softplus else 1)
    return dict(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(dy * x).sum((0, 1)), dbias=ddt.sum((0, 1)), dz=dz, dh0=dh)


# ---- cache ---------------------------------------------------------------------------------------------
def cache(v, group, fmt):
    """(values read back before their last rounding, scales) by exact arithmetic in 64 bits."""
    flat = d64(v).reshape(v.shape[0], -1, group)
    most = 127.0 if fmt == "int8" else 448.0
    big = flat.abs().amax(-1)
    scale = (big / most).float().double()
    scale = torch.where(scale < 2.0 ** -80, torch.zeros_like(scale), scale)
    q = flat / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    q = torch.where(scale[..., None] > 0, q, torch.zeros_like(q)).clamp(-most, most)
    if fmt == "int8":
        code = q.round()
    else:
        step = 2.0 ** (torch.frexp(q).exponent.clamp(min=-5).double() - 4)
        code = (q / step).round() * step
    bad = ~torch.isfinite(big)
    scale = torch.where(bad, torch.full_like(scale, float("nan")), scale)
    return (code * scale[..., None]).reshape(v.shape), scale
