"""Measured cases of the selective-scan operators: the short causal convolution, the selective
state space scan (prompts, training, single tokens) and the 8-bit state cache.

``run`` computes a case in its plain form (elementary torch operations in fp32), or, with ``own``
set, through mamba_ssd_prefill_amd.  Shapes are those of the repository's Mamba-2 130M and 2.7B
layers (inner widths 1536 and 5120; 1792 and 5376 convolution channels) with 16 states a channel,
and generic ones.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}
DEV = "cuda"


def listed():
    """4 to 12 cases; each comment says what it stands for."""
    return [
        # one generated token of one user through the 2.7B block's convolution: latency counts
        dict(name="conv step 1 row", op="conv_step", batch=1, channels=5376, width=4, dtype="bf16", slots=1),
        # a packed prompt batch of mixed lengths, each sequence with its own state, 130M block
        dict(name="conv prompt packed", op="conv_prompt", batch=1, seqlen=4096, channels=1792, width=4, dtype="f16",
             nseq=9),
        # one training step's convolution, 2.7B block
        dict(name="conv training", op="conv_train", batch=2, seqlen=4096, channels=5376, width=4, dtype="bf16"),
        # one generated token of one user, 130M layer
        dict(name="scan step 1 row", op="scan_step", batch=1, channels=1536, dstate=16, groups=1, dtype="bf16",
             state="f32", slots=1),
        # one generated token for a full serving batch, 2.7B layer, states in a pool
        dict(name="scan step 256 rows", op="scan_step", batch=256, channels=5120, dstate=16, groups=1, dtype="bf16",
             state="f32", slots=288),
        # a short chat turn continuing a cached state
        dict(name="scan prompt short", op="scan_prompt", batch=1, seqlen=131, channels=1536, dstate=16, groups=1,
             dtype="f16", state="f32", nseq=0, gate=True),
        # packed prompts of odd lengths in fp32, two B/C groups, an odd width
        dict(name="scan prompt packed f32", op="scan_prompt", batch=1, seqlen=3001, channels=1110, dstate=32, groups=2,
             dtype="f32", state="f32", nseq=7, gate=False),
        # long documents, 2.7B layer
        dict(name="scan prompt long", op="scan_prompt", batch=2, seqlen=8192, channels=5120, dstate=16, groups=1,
             dtype="bf16", state="f32", nseq=0, gate=True),
        # a small training step, 130M layer
        dict(name="scan training small", op="scan_train", batch=2, seqlen=500, channels=1536, dstate=16, groups=1,
             dtype="f16", gate=True),
        # a training step of the 2.7B layer
        dict(name="scan training", op="scan_train", batch=2, seqlen=2048, channels=5120, dstate=16, groups=1,
             dtype="bf16", gate=True),
        # the states of 16 finished prompts (2.7B Mamba-2 layer) put into the 8-bit pool and read back
        dict(name="cache int8 2.7B", op="cache", batch=16, rows=5120, dstate=128, group=128, state="f32",
             format="int8", slots=24),
        # one prompt's scan state, 130M layer, 8-bit floating point
        dict(name="cache e4m3 one prompt", op="cache", batch=1, rows=1536, dstate=16, group=16, state="f16",
             format="e4m3", slots=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["conv_step", "conv_prompt", "conv_train", "scan_step", "scan_prompt", "scan_train", "cache"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    state = rng.choice(["f32", "f32", "f16", "bf16"])
    channels = _log(rng, 64, 5376)
    if op == "conv_step":
        batch = _log(rng, 1, 256)
        return dict(op=op, batch=batch, channels=channels, width=rng.choice([2, 3, 4]), dtype=dtype,
                    slots=batch + rng.randint(0, 32))
    if op in ("conv_prompt", "conv_train"):
        batch = _log(rng, 1, 4)
        seqlen = max(1, min(_log(rng, 4, 8192), 2 * 4096 * 5376 // (batch * channels)))
        c = dict(op=op, batch=batch, seqlen=seqlen, channels=channels, width=rng.choice([2, 3, 4]), dtype=dtype)
        if op == "conv_prompt":
            c["nseq"] = rng.choice([0, batch * min(seqlen, rng.randint(1, 12))])
        return c
    groups = rng.choice([1, 1, 2, 4])
    channels = groups * max(1, channels // groups)
    dstate = rng.choice([8, 16, 16, 32, 64])
    if op == "scan_step":
        batch = max(1, min(_log(rng, 1, 256), 256 * 5120 * 16 // (channels * dstate)))
        return dict(op=op, batch=batch, channels=channels, dstate=dstate, groups=groups, dtype=dtype, state=state,
                    slots=batch + rng.randint(0, 32))
    if op in ("scan_prompt", "scan_train"):
        most = 2 * 8192 * 5120 * 16 if op == "scan_prompt" else 2 * 2048 * 5120 * 16
        batch = _log(rng, 1, 8)
        seqlen = max(1, min(_log(rng, 4, 8192), most // (batch * channels * dstate)))
        c = dict(op=op, batch=batch, seqlen=seqlen, channels=channels, dstate=dstate, groups=groups, dtype=dtype,
                 gate=rng.random() < 0.6)
        if op == "scan_prompt":
            c.update(state=state, nseq=rng.choice([0, batch * min(seqlen, rng.randint(1, 12))]))
        return c
    dstate = rng.choice([16, 32, 64, 128])
    rows = 8 * _log(rng, 8, 640)
    batch = max(1, min(_log(rng, 1, 64), 16 * 5120 * 128 // (rows * dstate)))
    return dict(op=op, batch=batch, rows=rows, dstate=dstate, group=rng.choice([16, 32, 64, 128]), state=state,
                format=rng.choice(["int8", "e4m3"]), slots=batch + rng.randint(0, 16))


def _cuts(case, seed):
    """Packed input: each batch row's sequences as (number, first token, length), and the row's
    tokens behind its last sequence are padding (number -1).  A row holds nseq / batch sequences."""
    rng = random.Random(seed * 1000003 + 17)
    B, L, per = case["batch"], case["seqlen"], case["nseq"] // case["batch"]
    rows = []
    for b in range(B):
        used = max(per, L - rng.randint(0, max(1, L // 32)))
        at = [0] + sorted(rng.sample(range(1, used), per - 1)) + [used]
        rows.append([(b * per + i, at[i], at[i + 1] - at[i]) for i in range(per)])
    return rows


def _packing(case, seed, s):
    s["nseq"] = case.get("nseq", 0)
    if not s["nseq"]:
        s["seq_idx"] = None
        return
    seq = torch.full((case["batch"], case["seqlen"]), -1, dtype=torch.int32)
    for b, row in enumerate(_cuts(case, seed)):
        for q, t0, n in row:
            seq[b, t0:t0 + n] = q
    s["seq_idx"] = seq.to(DEV)
    # the plan that the program packed by: each sequence's first and last token (over all rows), each
    # token's place in its sequence, and whether it goes on from the token before it
    cuts = [(b, t0, n) for b, row in enumerate(_cuts(case, seed)) for _, t0, n in row]
    L = case["seqlen"]
    s["first"] = torch.tensor([b * L + t0 for b, t0, n in cuts], device=DEV)
    s["last"] = torch.tensor([b * L + t0 + n - 1 for b, t0, n in cuts], device=DEV)
    inside = torch.ones(case["batch"], L)
    inside[:, 0] = 0
    inside[:, 1:][seq[:, 1:] != seq[:, :-1]] = 0
    t = torch.arange(L).expand(case["batch"], L)
    s["pos"] = (t - torch.where(inside == 0, t, 0).cummax(1).values).to(DEV)
    s["inside"] = inside.to(DEV)


def prepare(case, seed):
    """Inputs of the case on the GPU: normal activations, steps of 1e-3 .. 1e-1 before their own
    variation, decays of -1 .. -N, as such layers hold them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    s = dict(case)
    op = case["op"]
    if op == "cache":
        st = DT[case["state"]]
        E = case["rows"] * case["dstate"]
        # a state's rows differ in size by orders of magnitude
        size = torch.exp(1.5 * rn(case["batch"], case["rows"], 1))
        s["value"] = (size * rn(case["batch"], case["rows"], case["dstate"])).to(st)
        s["index"] = torch.randperm(case["slots"], generator=g, device=DEV)[:case["batch"]].to(torch.int32)
        code = torch.int8 if case["format"] == "int8" else torch.float8_e4m3fn
        s["codes"] = torch.zeros(case["slots"], case["rows"], case["dstate"], dtype=code, device=DEV)
        s["scales"] = torch.zeros(case["slots"], E // case["group"], dtype=torch.float32, device=DEV)
        return s
    dt_, Ch, Bt = DT[case["dtype"]], case["channels"], case["batch"]
    L = case.get("seqlen")
    lead = (Bt,) if L is None else (Bt, L)
    if op.startswith("conv"):
        W = case["width"]
        s["x"] = rn(*lead, Ch).to(dt_)
        s["w"] = 0.5 * rn(Ch, W)
        s["b"] = 0.1 * rn(Ch)
        if op == "conv_train":
            s["dout"] = rn(*lead, Ch).to(dt_)
        elif op == "conv_prompt":
            _packing(case, seed, s)
            s["h0"] = rn(s["nseq"] or Bt, Ch, W - 1).to(dt_)
        else:
            s["pool"] = rn(case["slots"], Ch, W - 1).to(dt_)
            s["index"] = torch.randperm(case["slots"], generator=g, device=DEV)[:Bt].to(torch.int32)
        return s
    N, G = case["dstate"], case["groups"]
    s["x"] = rn(*lead, Ch).to(dt_)
    s["dt"] = (0.5 * rn(*lead, Ch)).to(dt_)
    target = torch.exp(math.log(1e-3) + torch.rand(Ch, generator=g, device=DEV) * (math.log(1e-1) - math.log(1e-3)))
    s["bias"] = target + torch.log(-torch.expm1(-target))
    s["A"] = -torch.arange(1, N + 1, device=DEV).float() * torch.exp(0.1 * rn(Ch, N))
    s["B"], s["C"] = rn(*lead, G, N).to(dt_), rn(*lead, G, N).to(dt_)
    s["D"] = rn(Ch)
    s["z"] = rn(*lead, Ch).to(dt_) if case.get("gate", True) else None
    if op == "scan_train":
        s["dout"] = rn(*lead, Ch).to(dt_)
    elif op == "scan_prompt":
        _packing(case, seed, s)
        s["h0"] = (0.5 * rn(s["nseq"] or Bt, Ch, N)).to(DT[case["state"]])
    else:
        s["pool"] = (0.5 * rn(case["slots"], Ch, N)).to(DT[case["state"]])
        s["index"] = torch.randperm(case["slots"], generator=g, device=DEV)[:Bt].to(torch.int32)
    return s


def run(s):
    if own:
        import mamba_ssd_prefill_amd as ssd
        return OWN[s["op"]](ssd, s)
    return PLAIN[s["op"]](s)


# ---- through the framework ----------------------------------------------------------------------
def _own_conv_prompt(ssd, s):
    return ssd.causal_conv(s["x"], s["w"], s["b"], initial_state=s["h0"], seq_idx=s["seq_idx"], nseq=s["nseq"] or None)


def _own_conv_train(ssd, s):
    out, _ = ssd.causal_conv(s["x"], s["w"], s["b"], with_final_state=False)
    g = ssd.causal_conv_backward(s["dout"], s["x"], s["w"], s["b"])
    return out, g.dx, g.dweight, g.dbias


def _own_conv_step(ssd, s):
    out = ssd.causal_conv_step(s["x"], s["w"], s["b"], state=s["pool"], slots=s["index"])
    return out, s["pool"]


def _own_scan_prompt(ssd, s):
    return ssd.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["bias"], s["z"],
                              initial_state=s["h0"], seq_idx=s["seq_idx"], nseq=s["nseq"] or None)


def _own_scan_train(ssd, s):
    out, _, saved = ssd.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["bias"], s["z"],
                                       save_for_backward=True)
    g = ssd.selective_scan_backward(s["dout"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["bias"], s["z"],
                                    saved=saved)
    return dict(out=out, dx=g.dx, ddt=g.ddt, dA=g.dA, dB=g.dB, dC=g.dC, dD=g.dD, dbias=g.ddt_bias, dz=g.dz)


def _own_scan_step(ssd, s):
    out = ssd.selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["bias"], s["z"],
                                  state=s["pool"], slots=s["index"])
    return out, s["pool"]


def _own_cache(ssd, s):
    ssd.state_cache_write(s["value"], s["codes"], s["scales"], s["index"])
    return ssd.state_cache_read(s["codes"], s["scales"], s["index"], state_dtype=s["value"].dtype), s["scales"]


OWN = dict(conv_prompt=_own_conv_prompt, conv_train=_own_conv_train, conv_step=_own_conv_step,
           scan_prompt=_own_scan_prompt, scan_train=_own_scan_train, scan_step=_own_scan_step, cache=_own_cache)


# ---- plain forms --------------------------------------------------------------------------------
def _silu(v):
    return v / (1 + torch.exp(-v))


def _dsilu(v):
    """The derivative of silu."""
    p = 1 / (1 + torch.exp(-v))
    return p * (1 + v * (1 - p))


def _plain_conv_prompt(s):
    x, w, h0 = s["x"].float(), s["w"], s["h0"].float()
    (Bt, L, Ch), W = x.shape, w.shape[1]
    if s["seq_idx"] is None:
        xp = torch.cat([h0.transpose(1, 2), x], 1)                        # [B, W-1+L, Ch]
        pre = (xp.unfold(1, W, 1) * w).sum(-1) + s["b"]
        return _silu(pre).to(s["x"].dtype), xp[:, L:].transpose(1, 2).to(s["x"].dtype).contiguous()
    # packed: tap k of a token p places into its sequence is the state's column p + k while p + k < W-1
    first, last, pos, seq = s["first"], s["last"], s["pos"], s["seq_idx"].long()
    place = pos[..., None] + torch.arange(W, device=x.device)             # [B, L, W]
    here = place >= W - 1
    t = (torch.arange(L, device=x.device)[:, None] + torch.arange(W, device=x.device) - (W - 1)).clamp(min=0)
    taps = x[:, t]                                                        # [B, L, W, Ch]
    old = h0[seq.clamp(min=0)[..., None], :, place.clamp(max=W - 2)]      # [B, L, W, Ch]
    old = torch.where((seq >= 0)[..., None, None], old, torch.zeros((), device=x.device))
    pre = (torch.where(here[..., None], taps, old) * w.t()).sum(2) + s["b"]
    n = last - first + 1
    back = n[:, None] + torch.arange(W - 1, device=x.device)              # [nseq, W-1]: place + W-1 of each kept input
    row = (first[:, None] + back - (W - 1)).clamp(min=0)
    kept = torch.where((back >= W - 1)[..., None], x.reshape(Bt * L, Ch)[row],
                       h0.transpose(1, 2).gather(1, back.clamp(max=W - 2)[..., None].expand(-1, -1, Ch)))
    return _silu(pre).to(s["x"].dtype), kept.transpose(1, 2).to(s["x"].dtype).contiguous()


def _plain_conv_train(s):
    x, w, dout = s["x"].float(), s["w"], s["dout"].float()
    W = w.shape[1]
    zeros = x.new_zeros(x.shape[0], W - 1, x.shape[2])
    taps = torch.cat([zeros, x], 1).unfold(1, W, 1)                       # [B, L, Ch, W]
    pre = (taps * w).sum(-1) + s["b"]
    dpre = dout * _dsilu(pre)
    dx = (torch.cat([dpre, zeros], 1).unfold(1, W, 1) * w.flip(1)).sum(-1)
    dw = (taps * dpre[..., None]).sum((0, 1))
    dt_ = s["x"].dtype
    return _silu(pre).to(dt_), dx.to(dt_), dw, dpre.sum((0, 1))


def _plain_conv_step(s):
    rows = s["index"].long()
    win = torch.cat([s["pool"][rows], s["x"][..., None]], -1)             # [B, Ch, W]
    pre = (win.float() * s["w"]).sum(-1) + s["b"]
    s["pool"][rows] = win[..., 1:]
    return _silu(pre).to(s["x"].dtype), s["pool"]


def _channels(v, Ch):
    """[..., G, N] -> [..., Ch, N]: each channel's row of its group."""
    v = v.float()
    return v[..., :, None, :].expand(*v.shape[:-1], Ch // v.shape[-2], v.shape[-1]).reshape(*v.shape[:-2], Ch, -1)


def _steps(s):
    v = s["dt"].float() + s["bias"]
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _scan(a, b):
    """h[t] = a[t] h[t-1] + b[t] along dimension 1 in log2(L) passes, each joining every stretch of
    tokens with the one of the same length before it."""
    n = 1
    while n < a.shape[1]:
        b = torch.cat([b[:, :n], torch.addcmul(b[:, n:], a[:, n:], b[:, :-n])], 1)
        if 2 * n < a.shape[1]:
            a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _plain_scan_prompt(s):
    x, A = s["x"].float(), s["A"]
    Bt, L, Ch = x.shape
    d = _steps(s)
    a = torch.exp(d[..., None] * A)
    b = (d * x)[..., None] * _channels(s["B"], Ch)
    h0 = s["h0"].float()
    if s["seq_idx"] is None:
        b[:, 0] += a[:, 0] * h0
        last = torch.arange(1, Bt + 1, device=x.device) * L - 1
    else:
        first, last = s["first"], s["last"]
        b.view(Bt * L, Ch, -1)[first] += a.view(Bt * L, Ch, -1)[first] * h0
        a = a * s["inside"][..., None, None]
    h = _scan(a, b)
    y = (h * _channels(s["C"], Ch)).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(s["x"].dtype), h.reshape(Bt * L, Ch, -1)[last].to(s["h0"].dtype)


def _plain_scan_train(s):
    x, A, D = s["x"].float(), s["A"], s["D"]
    Bt, L, Ch = x.shape
    G, N = s["B"].shape[2:]
    dtype = s["x"].dtype
    v = s["dt"].float() + s["bias"]
    d = _steps(s)
    B, C = _channels(s["B"], Ch), _channels(s["C"], Ch)
    a = torch.exp(d[..., None] * A)
    h = _scan(a, (d * x)[..., None] * B)
    y = (h * C).sum(-1) + D * x
    dout = s["dout"].float()
    if s["z"] is None:
        out, dy, dz = y, dout, None
    else:
        z = s["z"].float()
        out, dy, dz = y * _silu(z), dout * _silu(z), (dout * y * _dsilu(z)).to(dtype)
    over = lambda t: t.view(Bt, L, G, Ch // G, N).sum(3).to(dtype)  # noqa: E731
    dC = over(dy[..., None] * h)
    # the gradient of h runs from the last token to the first
    g = _scan(torch.cat([a.new_zeros(Bt, 1, Ch, N), a[:, 1:].flip(1)], 1), (dy[..., None] * C).flip(1)).flip(1)
    dB = over(g * (d * x)[..., None])
    sB = (g * B).sum(-1)
    q = g * a * torch.cat([h.new_zeros(Bt, 1, Ch, N), h[:, :-1]], 1)
    ddt = (x * sB + (q * A).sum(-1)) / (1 + torch.exp(-v))
    return dict(out=out.to(dtype), dx=(D * dy + d * sB).to(dtype), ddt=ddt.to(dtype), dA=(d[..., None] * q).sum((0, 1)),
                dB=dB, dC=dC, dD=(dy * x).sum((0, 1)), dbias=ddt.sum((0, 1)), dz=dz)


def _plain_scan_step(s):
    rows, x = s["index"].long(), s["x"].float()
    Ch = x.shape[1]
    d = _steps(s)[..., None]
    h = torch.exp(d * s["A"]) * s["pool"][rows].float() + d * x[..., None] * _channels(s["B"], Ch)
    y = (h * _channels(s["C"], Ch)).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["pool"][rows] = h.to(s["pool"].dtype)
    return y.to(s["x"].dtype), s["pool"]


def _plain_cache(s):
    # 64 bits: quotients next to the border between two codes
    v = s["value"].double().view(s["batch"], -1, s["group"])
    most = 127.0 if s["format"] == "int8" else 448.0
    scale = (v.abs().amax(-1, keepdim=True) / most).float()
    q = v / torch.where(scale > 0, scale, 1.0).double()
    if s["format"] == "int8":
        code = q.round().clamp(-127, 127)
    else:
        # steps of 2^-3 of the power of two below |q|, and of 2^-9 below 2^-6
        step = torch.ldexp(torch.ones_like(q), torch.frexp(q).exponent.clamp(min=-5) - 4)
        code = ((q / step).round() * step).clamp(-448, 448)
    scale = torch.where(scale > 0, scale, 0.0)
    s["scales"][s["index"].long()] = scale[..., 0]
    return (code.float() * scale).view(s["value"].shape).to(s["value"].dtype), s["scales"]


PLAIN = dict(conv_prompt=_plain_conv_prompt, conv_train=_plain_conv_train, conv_step=_plain_conv_step,
             scan_prompt=_plain_scan_prompt, scan_train=_plain_scan_train, scan_step=_plain_scan_step,
             cache=_plain_cache)


# ---- in 64 bits, from the definitions -----------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return EXACT[case["op"]](s, case, seed)


def _rows(s, case, seed):
    """(batch row, number of the state, first token, tokens) of every sequence, the padding with -1."""
    if not s["nseq"]:
        return [(b, b, 0, case["seqlen"]) for b in range(case["batch"])]
    out = []
    for b, row in enumerate(_cuts(case, seed)):
        end = row[-1][1] + row[-1][2]
        out += [(b, q, t0, n) for q, t0, n in row]
        out += [(b, -1, end, case["seqlen"] - end)] if end < case["seqlen"] else []
    return out


def _gate64(v):
    return v * torch.sigmoid(v)


def _exact_conv_prompt(s, case, seed):
    x, w = s["x"].double(), s["w"].double()
    W = w.shape[1]
    out, fin = torch.zeros_like(x), torch.zeros_like(s["h0"], dtype=torch.float64)
    for b, q, t0, n in _rows(s, case, seed):
        old = s["h0"][q].double() if q >= 0 else x.new_zeros(x.shape[2], W - 1)
        seq = torch.cat([old.t(), x[b, t0:t0 + n]])                       # [W-1+n, Ch]
        pre = s["b"].double().expand(n, -1).clone()
        for k in range(W):
            pre += seq[k:k + n] * w[:, k]
        out[b, t0:t0 + n] = _gate64(pre)
        if q >= 0:
            fin[q] = seq[n:].t()
    return out, fin


def _exact_conv_train(s, case, seed):
    x, w, b = (s[k].double().requires_grad_() for k in ("x", "w", "b"))
    W, L = w.shape[1], x.shape[1]
    xp = torch.cat([x.new_zeros(x.shape[0], W - 1, x.shape[2]), x], 1)
    pre = sum(xp[:, k:k + L] * w[:, k] for k in range(W)) + b
    out = _gate64(pre)
    dx, dw, db = torch.autograd.grad(out, (x, w, b), s["dout"].double())
    return out.detach(), dx, dw, db


def _exact_conv_step(s, case, seed):
    pool = s["pool"].double()
    rows = s["index"].long()
    win = torch.cat([pool[rows], s["x"].double()[:, :, None]], 2)
    pre = torch.einsum("bcw,cw->bc", win, s["w"].double()) + s["b"].double()
    pool[rows] = win[:, :, 1:]
    return _gate64(pre), pool


def _spread(v, Ch):
    return v.double().repeat_interleave(Ch // v.shape[-2], dim=-2)


def _exact_scan_prompt(s, case, seed):
    x, A = s["x"].double(), s["A"].double()
    d = torch.logaddexp(s["dt"].double() + s["bias"].double(), x.new_zeros(()))
    Ch = x.shape[2]
    y, fin = torch.zeros_like(x), torch.zeros_like(s["h0"], dtype=torch.float64)
    rows = _rows(s, case, seed)
    # rows of one length go through the recurrence together, token by token
    groups = [rows] if not s["nseq"] else [[r] for r in rows]
    for grp in groups:
        bs, t0, n = [r[0] for r in grp], grp[0][2], grp[0][3]
        live = [i for i, r in enumerate(grp) if r[1] >= 0]
        h = x.new_zeros(len(grp), Ch, A.shape[1])
        for i in live:
            h[i] = s["h0"][grp[i][1]].double()
        for t in range(t0, t0 + n):
            dt_ = d[bs, t][..., None]
            h = torch.exp(dt_ * A) * h + dt_ * x[bs, t][..., None] * _spread(s["B"][bs, t], Ch)
            y[bs, t] = (h * _spread(s["C"][bs, t], Ch)).sum(-1)
        for i in live:
            fin[grp[i][1]] = h[i]
    y = y + s["D"].double() * x
    return (y if s["z"] is None else y * _gate64(s["z"].double())), fin


def _exact_scan_train(s, case, seed):
    x, A, D = s["x"].double(), s["A"].double(), s["D"].double()
    Bt, L, Ch = x.shape
    G, N = s["B"].shape[2:]
    v = s["dt"].double() + s["bias"].double()
    d = torch.logaddexp(v, x.new_zeros(()))
    hs = torch.zeros(L + 1, Bt, Ch, N, dtype=torch.float64, device=x.device)
    y = torch.zeros_like(x)
    for t in range(L):
        dt_ = d[:, t, :, None]
        hs[t + 1] = torch.exp(dt_ * A) * hs[t] + dt_ * x[:, t, :, None] * _spread(s["B"][:, t], Ch)
        y[:, t] = (hs[t + 1] * _spread(s["C"][:, t], Ch)).sum(-1)
    y = y + D * x
    dout = s["dout"].double()
    if s["z"] is None:
        out, dy, dz = y, dout, None
    else:
        z = s["z"].double().requires_grad_()
        gate = _gate64(z)
        dz, = torch.autograd.grad(gate, z, dout * y)
        gate = gate.detach()
        out, dy = y * gate, dout * gate
    dB, dC = (torch.zeros(Bt, L, G, N, dtype=torch.float64, device=x.device) for _ in range(2))
    dx, dd, dA, carry = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(A), torch.zeros_like(hs[0])
    for t in reversed(range(L)):
        dt_, u = d[:, t, :, None], x[:, t, :, None]
        B = _spread(s["B"][:, t], Ch)
        g = carry + dy[:, t, :, None] * _spread(s["C"][:, t], Ch)
        dC[:, t] = (dy[:, t, :, None] * hs[t + 1]).view(Bt, G, -1, N).sum(2)
        dB[:, t] = (g * dt_ * u).view(Bt, G, -1, N).sum(2)
        dx[:, t] = (g * dt_ * B).sum(-1)
        carry = g * torch.exp(dt_ * A)
        dexp = carry * hs[t]                                              # gradient of the exponent
        dA += (dexp * dt_).sum(0)
        dd[:, t] = (g * u * B + dexp * A).sum(-1)
    ddt = dd * torch.sigmoid(v)
    return dict(out=out, dx=dx + D * dy, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(dy * x).sum((0, 1)), dbias=ddt.sum((0, 1)),
                dz=dz)


def _exact_scan_step(s, case, seed):
    pool, rows, x = s["pool"].double(), s["index"].long(), s["x"].double()
    Ch = x.shape[1]
    d = torch.logaddexp(s["dt"].double() + s["bias"].double(), x.new_zeros(()))
    h = torch.exp(d[..., None] * s["A"].double()) * pool[rows]
    h += (d * x)[..., None] * _spread(s["B"], Ch)
    y = torch.einsum("bcn,bcn->bc", h, _spread(s["C"], Ch)) + s["D"].double() * x
    pool[rows] = h
    return (y if s["z"] is None else y * _gate64(s["z"].double())), pool


def _exact_cache(s, case, seed):
    v = s["value"].double().flatten(1).unflatten(1, (-1, case["group"]))
    if case["format"] == "int8":
        grid = torch.arange(-127, 128, device=DEV).double()
        most = 127
    else:  # every value of four exponent bits (bias 7) and three mantissa bits but NaN
        grid = torch.tensor([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                             for e in range(16) for m in range(8)][:-1], dtype=torch.float64, device=DEV)
        grid = torch.cat([-grid.flip(0)[:-1], grid])
        most = 448
    scale = (v.abs().amax(-1) / most).float().double()                    # the scale is held in fp32
    q = (v / scale.clamp(min=1e-300)[..., None]).clamp(-most, most)
    hi = torch.searchsorted(grid, q.contiguous()).clamp(1, grid.numel() - 1)
    up, down = grid[hi] - q, q - grid[hi - 1]
    # the codes' order on the grid is their order as numbers, so ties go to the even index from zero
    even = (hi - grid.numel() // 2) % 2 == 0
    take = (up < down) | ((up == down) & even)
    near = torch.where(take, grid[hi], grid[hi - 1])
    scales = s["scales"].double()
    scales[s["index"].long()] = scale
    return (near * scale[..., None]).view(s["value"].shape), scales


EXACT = dict(conv_prompt=_exact_conv_prompt, conv_train=_exact_conv_train, conv_step=_exact_conv_step,
             scan_prompt=_exact_scan_prompt, scan_train=_exact_scan_train, scan_step=_exact_scan_step,
             cache=_exact_cache)


def work(case):
    """Bytes that have to move and operations that have to be done in one pass."""
    op = case["op"]
    if op == "cache":
        n = case["batch"] * case["rows"] * case["dstate"]
        st = ES[case["state"]]
        # written: read the state, write codes and scales; read back: the reverse
        return {"bytes": n * 2 * (st + 1 + 4 / case["group"]), "flops": 5 * n}
    e, Ch, Bt = ES[case["dtype"]], case["channels"], case["batch"]
    tokens = Bt * case.get("seqlen", 1)
    if op.startswith("conv"):
        W = case["width"]
        w = Ch * (W + 1) * 4
        n = tokens * Ch
        if op == "conv_step":
            return {"bytes": n * e * (2 + 2 * (W - 1)) + w, "flops": n * (2 * W + 4)}
        if op == "conv_prompt":
            states = 2 * (case["nseq"] or Bt) * Ch * (W - 1) * e
            return {"bytes": 2 * n * e + w + states + (4 * tokens if case["nseq"] else 0), "flops": n * (2 * W + 4)}
        # out from x; dx, dw and db from x and dout
        return {"bytes": 5 * n * e + 3 * w, "flops": n * (8 * W + 14)}
    N, G = case["dstate"], case["groups"]
    n = tokens * Ch
    par = Ch * (N + 2) * 4
    rows = 2 * tokens * G * N * e
    gate = 1 if case.get("gate", True) else 0
    if op == "scan_step":
        return {"bytes": 2 * n * N * ES[case["state"]] + 4 * n * e + rows + par, "flops": n * (7 * N + 12)}
    if op == "scan_prompt":
        states = 2 * (case["nseq"] or Bt) * Ch * N * ES[case["state"]]
        return {"bytes": (3 + gate) * n * e + rows + par + states, "flops": n * (7 * N + 12)}
    # forward: x, dt, z -> out; backward: x, dt, z, dout -> dx, ddt, dz; B, C twice and their gradients
    return {"bytes": (3 + gate + 5 + 2 * gate) * n * e + 3 * rows + 3 * par, "flops": n * (7 * N + 12 + 21 * N + 40)}
