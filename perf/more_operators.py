"""Measured cases of a recurrent layer's other operators: the root-mean-square norm with the residual's addition (and an
8-bit output), the matrix product with bias, activation and residual, and the gated linear recurrence.

``run`` computes a case in its plain form (elementary torch operations in fp32), or, with ``own`` set, through
mamba_ssd_prefill_amd.  Shapes are those of the repository's Mamba-2 130M and 2.7B layers (inner widths 1536 and
5120, model widths half of that, a joint projection of 10576 outputs), and generic ones.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}
DEV = "cuda"
EPS = 1e-5


def listed():
    """4 to 12 cases; each comment says what it stands for."""
    return [
        # the norm before a layer, one generated token of one user, 2.7B: latency counts
        dict(name="norm 1 token", op="norm", rows=1, width=2560, dtype="bf16", residual="same"),
        # a training step's norm, 2.7B, residual stream in fp32
        dict(name="norm training", op="norm_train", rows=2 * 4096, width=2560, dtype="bf16", residual="f32"),
        # a prompt's norm and joint projection in 8 bits, 2.7B
        dict(name="norm + product e4m3", op="norm_product8", rows=2048, width=2560, outs=10576, dtype="bf16",
             residual="same", format="e4m3"),
        # one generated token for 32 users: norm and a projection of odd width in 8 bits
        dict(name="norm + product int8 32 rows", op="norm_product8", rows=32, width=1536, outs=771, dtype="f16",
             residual="same", format="int8"),
        # the joint projection of one generated token, 2.7B
        dict(name="product 1 token", op="product", rows=1, width=2560, outs=10576, dtype="bf16", bias=False, act="",
             residual=False),
        # the projection back to the residual stream, long prompts, 2.7B
        dict(name="product prompt", op="product", rows=8192, width=5120, outs=2560, dtype="bf16", bias=False, act="",
             residual=True),
        # odd sizes everywhere, fp32
        dict(name="product ragged f32", op="product", rows=333, width=1110, outs=771, dtype="f32", bias=True, act="gelu",
             residual=True),
        # the backward pass of a layer's widening projection
        dict(name="product training", op="product_train", rows=4096, width=1024, outs=4096, dtype="f16", bias=True,
             act="silu"),
        # one generated token for a full serving batch, 2.7B width, states in a pool
        dict(name="recurrence step 256 rows", op="rec_step", batch=256, channels=5120, dtype="bf16", state="f32",
             slots=288, in_gate=True, normalize=True),
        # packed prompts of odd lengths in fp32, an odd width, each with its own state
        dict(name="recurrence packed f32", op="rec_prompt", batch=1, seqlen=3001, channels=1110, dtype="f32", state="f32",
             nseq=7, in_gate=True, normalize=True),
        # long documents, 2.7B width
        dict(name="recurrence long", op="rec_prompt", batch=2, seqlen=8192, channels=5120, dtype="bf16", state="f32",
             nseq=0, in_gate=True, normalize=True),
        # a training step, 2.7B width
        dict(name="recurrence training", op="rec_train", batch=2, seqlen=4096, channels=5120, dtype="bf16", in_gate=True,
             normalize=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["norm", "norm_train", "norm_product8", "product", "product", "product_train", "rec_step",
                     "rec_prompt", "rec_train"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op.startswith("rec"):
        channels, gate, normalize = _log(rng, 64, 5376), rng.random() < 0.7, rng.random() < 0.7
        c = dict(op=op, channels=channels, dtype=dtype, in_gate=gate, normalize=normalize)
        if op == "rec_step":
            batch = _log(rng, 1, 256)
            return dict(c, batch=batch, state=rng.choice(["f32", "f32", "f16", "bf16"]), slots=batch + rng.randint(0, 32))
        most = (2 * 8192 if op == "rec_prompt" else 2 * 4096) * 5120
        batch = _log(rng, 1, 8)
        seqlen = max(1, min(_log(rng, 4, 8192), most // (batch * channels)))
        c.update(batch=batch, seqlen=seqlen)
        if op == "rec_prompt":
            c.update(state=rng.choice(["f32", "f32", "f16", "bf16"]),
                     nseq=rng.choice([0, batch * min(seqlen, rng.randint(1, 12))]))
        return c
    rows, width = _log(rng, 1, 8192), _log(rng, 64, 5376)
    if op in ("norm", "norm_train"):
        return dict(op=op, rows=rows, width=width, dtype=dtype, residual=rng.choice(["", "same", "f32"]))
    outs = _log(rng, 64, 10576)
    most = 8192 * 5120 * 2560 // (2 if op == "product_train" else 1)
    rows = max(1, min(rows, most // (width * outs)))
    if op == "norm_product8":
        return dict(op=op, rows=rows, width=width, outs=outs, dtype=rng.choice(["bf16", "f16"]),
                    residual=rng.choice(["", "same", "f32"]), format=rng.choice(["int8", "e4m3"]))
    c = dict(op=op, rows=rows, width=width, outs=outs, dtype=dtype, bias=rng.random() < 0.5,
             act=rng.choice(["", "silu", "gelu"]))
    if op == "product":
        c["residual"] = rng.random() < 0.5
    return c


def _cuts(case, seed):
    """Packed input: each batch row's sequences as (number, first token, length), and the row's tokens behind
    its last sequence are padding (number -1).  A row holds nseq / batch sequences."""
    rng = random.Random(seed * 1000003 + 29)
    B, L, per = case["batch"], case["seqlen"], case["nseq"] // case["batch"]
    rows = []
    for b in range(B):
        used = max(per, L - rng.randint(0, max(1, L // 32)))
        at = [0] + sorted(rng.sample(range(1, used), per - 1)) + [used]
        rows.append([(b * per + i, at[i], at[i + 1] - at[i]) for i in range(per)])
    return rows


def _packing(case, seed, s):
    s["nseq"] = case.get("nseq", 0)
    s["seq_idx"] = None
    if not s["nseq"]:
        return
    B, L = case["batch"], case["seqlen"]
    seq = torch.full((B, L), -1, dtype=torch.int32)
    cuts = [(b, q, t0, n) for b, row in enumerate(_cuts(case, seed)) for q, t0, n in row]
    for b, q, t0, n in cuts:
        seq[b, t0:t0 + n] = q
    s["seq_idx"] = seq.to(DEV)
    # the plan that the program packed by: first and last tokens over all rows, and whether a token goes on from the
    # one before it
    s["first"] = torch.tensor([b * L + t0 for b, _, t0, _ in cuts], device=DEV)
    s["last"] = torch.tensor([b * L + t0 + n - 1 for b, _, t0, n in cuts], device=DEV)
    inside = torch.ones(B, L)
    inside[:, 0] = 0
    inside[:, 1:][seq[:, 1:] != seq[:, :-1]] = 0
    s["inside"] = inside.to(DEV)


def prepare(case, seed):
    """Inputs of the case on the GPU: normal activations, weights of 1 / sqrt(width), decays of 0.9 to 0.999 a token at an
    open gate, as such layers hold them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    s = dict(case)
    op, dt_ = case["op"], DT[case["dtype"]]
    if op.startswith("norm"):
        M, K = case["rows"], case["width"]
        s["x"] = rn(M, K).to(dt_)
        s["res"] = {"": None, "same": dt_, "f32": torch.float32}[case["residual"]]
        if s["res"] is not None:
            s["res"] = (3 * rn(M, K)).to(s["res"])
        s["w"] = 1 + 0.2 * rn(K)
        if op == "norm_train":
            s["dout"] = rn(M, K).to(dt_)
            s["dsum"] = None if s["res"] is None else rn(M, K).to(s["res"].dtype)
        if op == "norm_product8":
            N = case["outs"]
            if case["format"] == "int8":
                s["wc"] = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
            else:
                s["wc"] = (100 * rn(N, K)).clamp(-448, 448).to(torch.float8_e4m3fn)
            s["ws"] = torch.exp(0.3 * rn(N)) / (100 * math.sqrt(K))
        return s
    if op.startswith("product"):
        M, K, N = case["rows"], case["width"], case["outs"]
        s["x"], s["w"] = rn(M, K).to(dt_), (rn(N, K) / math.sqrt(K)).to(dt_)
        s["b"] = 0.1 * rn(N) if case["bias"] else None
        s["res"] = rn(M, N).to(dt_) if case.get("residual") else None
        if op == "product_train":
            s["dout"] = rn(M, N).to(dt_)
            s["pre"] = rn(M, N).to(dt_) if case["act"] else None
        return s
    B, Ch = case["batch"], case["channels"]
    lead = (B, case["seqlen"]) if "seqlen" in case else (B,)
    s["x"], s["gate"] = rn(*lead, Ch).to(dt_), rn(*lead, Ch).to(dt_)
    s["ig"] = rn(*lead, Ch).to(dt_) if case["in_gate"] else None
    s["A"] = torch.log(0.9 + 0.099 * torch.rand(Ch, generator=g, device=DEV))
    s["gb"] = 0.5 * rn(Ch)
    s["ib"] = 0.5 * rn(Ch) if case["in_gate"] else None
    if op == "rec_train":
        s["dout"] = rn(*lead, Ch).to(dt_)
    elif op == "rec_prompt":
        _packing(case, seed, s)
        s["h0"] = rn(s["nseq"] or B, Ch).to(DT[case["state"]])
    else:
        s["pool"] = rn(case["slots"], Ch).to(DT[case["state"]])
        s["index"] = torch.randperm(case["slots"], generator=g, device=DEV)[:B].to(torch.int32)
    return s


def run(s):
    if own:
        import mamba_ssd_prefill_amd as ssd
        return OWN[s["op"]](ssd, s)
    return PLAIN[s["op"]](s)


# ---- through the framework ----------------------------------------------------------------------
def _own_norm(ssd, s):
    return ssd.rms_norm(s["x"], s["w"], s["res"], eps=EPS)


def _own_norm_train(ssd, s):
    out = ssd.rms_norm(s["x"], s["w"], s["res"], eps=EPS)
    out, total = (out, s["x"]) if s["res"] is None else out
    g = ssd.rms_norm_backward(s["dout"], total, s["w"], eps=EPS, dresidual=s["dsum"])
    return dict(out=out, sum=total, dx=g.dx, dres=g.dresidual, dw=g.dweight)


def _own_norm_product8(ssd, s):
    codes, scales, *total = ssd.rms_norm(s["x"], s["w"], s["res"], eps=EPS, format=s["format"])
    out = ssd.linear(codes, s["wc"], x_scale=scales, weight_scale=s["ws"], out_dtype=s["x"].dtype)
    return dict(out=out, scales=scales, sum=total)


def _own_product(ssd, s):
    return ssd.linear(s["x"], s["w"], s["b"], s["res"], activation=s["act"] or None)


def _own_product_train(ssd, s):
    g = ssd.linear_backward(s["dout"], s["x"], s["w"], pre=s["pre"], activation=s["act"] or None, with_bias=s["bias"])
    return dict(dx=g.dx, dw=g.dweight, db=g.dbias)


def _own_rec_step(ssd, s):
    out = ssd.gated_recurrence_step(s["x"], s["gate"], s["A"], s["ig"], s["gb"], s["ib"], state=s["pool"],
                                    slots=s["index"], normalize=s["normalize"])
    return out, s["pool"]


def _own_rec_prompt(ssd, s):
    return ssd.gated_recurrence(s["x"], s["gate"], s["A"], s["ig"], s["gb"], s["ib"], normalize=s["normalize"],
                                initial_state=s["h0"], seq_idx=s["seq_idx"], nseq=s["nseq"] or None)


def _own_rec_train(ssd, s):
    args = (s["x"], s["gate"], s["A"], s["ig"], s["gb"], s["ib"])
    out, _, saved = ssd.gated_recurrence(*args, normalize=s["normalize"], save_for_backward=True)
    g = ssd.gated_recurrence_backward(s["dout"], *args, saved=saved, normalize=s["normalize"])
    return dict(out=out, dx=g.dx, dgate=g.dgate, dA=g.dA, dig=g.din_gate, dgb=g.dgate_bias, dib=g.din_bias)


OWN = dict(norm=_own_norm, norm_train=_own_norm_train, norm_product8=_own_norm_product8, product=_own_product,
           product_train=_own_product_train, rec_step=_own_rec_step, rec_prompt=_own_rec_prompt, rec_train=_own_rec_train)


# ---- plain forms --------------------------------------------------------------------------------
def _total(s):
    return s["x"].float() if s["res"] is None else s["x"].float() + s["res"].float()


def _inverse_rms(t):
    return 1 / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    t = _total(s)
    out = (t * _inverse_rms(t) * s["w"]).to(s["x"].dtype)
    return out if s["res"] is None else (out, t.to(s["res"].dtype))


def _plain_norm_train(s):
    t = _total(s)
    out = (t * _inverse_rms(t) * s["w"]).to(s["x"].dtype)
    total = s["x"] if s["res"] is None else t.to(s["res"].dtype)
    t = total.float()                                                     # the gradients are those at the sum as kept
    inv = _inverse_rms(t)
    n, dout = t * inv, s["dout"].float()
    g = dout * s["w"]
    d = inv * (g - n * (g * n).mean(-1, keepdim=True))
    d = d if s["dsum"] is None else d + s["dsum"].float()
    return dict(out=out, sum=total, dx=d.to(s["x"].dtype), dres=d.to(total.dtype), dw=(dout * n).sum(0))


def _plain_norm_product8(s):
    t = _total(s).double()                                                # 64 bits: quotients next to the border of two codes
    y = t * _inverse_rms(t) * s["w"]
    most = 127.0 if s["format"] == "int8" else 448.0
    scales = (y.abs().amax(-1) / most).float()
    q = y / scales.double()[:, None]
    if s["format"] == "int8":
        codes = q.round()
    else:
        # steps of 2^-3 of the power of two below |q|, and of 2^-9 below 2^-6
        step = torch.ldexp(torch.ones_like(q), torch.frexp(q).exponent.clamp(min=-5) - 4)
        codes = ((q / step).round() * step).clamp(-448, 448)
    out = (codes.float() @ s["wc"].float().t()) * scales[:, None] * s["ws"]
    total = [] if s["res"] is None else [t.to(s["res"].dtype)]
    return dict(out=out.to(s["x"].dtype), scales=scales, sum=total)


def _gelu(v):
    return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))


def _silu(v):
    return v / (1 + torch.exp(-v))


def _plain_product(s):
    v = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        v = v + s["b"]
    v = _silu(v) if s["act"] == "silu" else _gelu(v) if s["act"] == "gelu" else v
    if s["res"] is not None:
        v = v + s["res"].float()
    return v.to(s["x"].dtype)


def _plain_product_train(s):
    d = s["dout"].float()
    if s["act"] == "silu":
        v = s["pre"].float()
        p = 1 / (1 + torch.exp(-v))
        d = d * p * (1 + v * (1 - p))
    elif s["act"] == "gelu":
        v = s["pre"].float()
        d = d * (0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi))
    t = s["x"].dtype
    return dict(dx=(d @ s["w"].float()).to(t), dw=(d.t() @ s["x"].float()).to(t), db=d.sum(0) if s["bias"] else None)


def _scan(a, b):
    """h[t] = a[t] h[t-1] + b[t] along dimension 1 in log2(L) passes, each joining every stretch of tokens with
    the one of the same length before it."""
    n = 1
    while n < a.shape[1]:
        b = torch.cat([b[:, :n], torch.addcmul(b[:, n:], a[:, n:], b[:, :-n])], 1)
        if 2 * n < a.shape[1]:
            a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _gates(s):
    """Gates r and i, decay a and the input's factor."""
    r = _sigmoid(s["gate"].float() + s["gb"])
    i = None if s["ig"] is None else _sigmoid(s["ig"].float() + s["ib"])
    l = r * s["A"]
    return r, i, torch.exp(l), torch.sqrt(-torch.expm1(2 * l)) if s["normalize"] else None


def _times(v, *factors):
    for f in factors:
        v = v if f is None else v * f
    return v


def _plain_rec_step(s):
    rows = s["index"].long()
    _, i, a, beta = _gates(s)
    h = a * s["pool"][rows].float() + _times(s["x"].float(), i, beta)
    s["pool"][rows] = h.to(s["pool"].dtype)
    return h.to(s["x"].dtype), s["pool"]


def _plain_rec_prompt(s):
    B, L, Ch = s["x"].shape
    _, i, a, beta = _gates(s)
    b, h0 = _times(s["x"].float(), i, beta), s["h0"].float()
    if s["seq_idx"] is None:
        b[:, 0] += a[:, 0] * h0
        last = torch.arange(1, B + 1, device=b.device) * L - 1
    else:
        last = s["last"]
        b.view(B * L, Ch)[s["first"]] += a.view(B * L, Ch)[s["first"]] * h0
        a = a * s["inside"][..., None]
    h = _scan(a, b)
    return h.to(s["x"].dtype), h.reshape(B * L, Ch)[last].to(s["h0"].dtype)


def _plain_rec_train(s):
    x, A = s["x"].float(), s["A"]
    B, L, Ch = x.shape
    r, i, a, beta = _gates(s)
    h = _scan(a, _times(x, i, beta))
    zero = a.new_zeros(B, 1, Ch)
    # the gradient of h runs from the last token to the first
    g = _scan(torch.cat([zero, a[:, 1:].flip(1)], 1), s["dout"].float().flip(1)).flip(1)
    dl = g * a * torch.cat([zero, h[:, :-1]], 1)
    if beta is not None:
        dl = dl - _times(g * x, i) * a * a / beta
    t = s["x"].dtype
    dgate = dl * A * r * (1 - r)
    dig = None if i is None else _times(g * x, beta) * i * (1 - i)
    return dict(out=h.to(t), dx=_times(g, i, beta).to(t), dgate=dgate.to(t), dA=(dl * r).sum((0, 1)),
                dig=None if dig is None else dig.to(t), dgb=dgate.sum((0, 1)), dib=None if dig is None else dig.sum((0, 1)))


PLAIN = dict(norm=_plain_norm, norm_train=_plain_norm_train, norm_product8=_plain_norm_product8, product=_plain_product,
             product_train=_plain_product_train, rec_step=_plain_rec_step, rec_prompt=_plain_rec_prompt,
             rec_train=_plain_rec_train)


# ---- in 64 bits, from the definitions -----------------------------------------------------------
def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed), case, seed)


def _exact_normed(x, res, w):
    v = x.double()
    if res is not None:
        v = v + res.double()
    return v, v * w.double() / torch.linalg.vector_norm(v, dim=1, keepdim=True).square().div(v.shape[1]).add(EPS).sqrt()


def _exact_norm(s, case, seed):
    v, y = _exact_normed(s["x"], s["res"], s["w"])
    return y if s["res"] is None else (y, v)


def _exact_norm_train(s, case, seed):
    v, y = _exact_normed(s["x"], s["res"], s["w"])
    kept = s["x"] if s["res"] is None else v.to(s["res"].dtype)           # what the backward pass is given
    k, w = kept.double().requires_grad_(), s["w"].double().requires_grad_()
    dk, dw = torch.autograd.grad(_exact_normed(k, None, w)[1], (k, w), s["dout"].double())
    if s["dsum"] is not None:
        dk = dk + s["dsum"].double()
    return dict(out=y, sum=v, dx=dk, dres=dk, dw=dw)


def _exact_norm_product8(s, case, seed):
    v, y = _exact_normed(s["x"], s["res"], s["w"])
    if case["format"] == "int8":
        grid = torch.arange(-127, 128, device=DEV).double()
    else:  # every value of four exponent bits (bias 7) and three mantissa bits but NaN
        grid = torch.tensor([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                             for e in range(16) for m in range(8)][:-1], dtype=torch.float64, device=DEV)
        grid = torch.cat([-grid.flip(0)[:-1], grid])
    scale = (y.abs().max(1).values / grid[-1]).float().double()           # the scale is held in fp32
    q = (y / scale[:, None]).clamp(grid[0], grid[-1]).contiguous()
    hi = torch.searchsorted(grid, q).clamp(1, grid.numel() - 1)
    up, down = grid[hi] - q, q - grid[hi - 1]
    # the codes' order on the grid is their order as numbers, so ties go to the even index from zero
    take = (up < down) | ((up == down) & ((hi - grid.numel() // 2) % 2 == 0))
    held = torch.where(take, grid[hi], grid[hi - 1]) * scale[:, None]
    out = torch.mm(held, (s["wc"].float().double() * s["ws"].double()[:, None]).T)
    return dict(out=out, scales=scale, sum=[] if s["res"] is None else [v])


def _act64(v, act):
    return v * torch.sigmoid(v) if act == "silu" else v * torch.special.ndtr(v) if act == "gelu" else v


def _exact_product(s, case, seed):
    v = torch.mm(s["x"].double(), s["w"].double().T)
    if case["bias"]:
        v += s["b"].double()
    v = _act64(v, case["act"])
    return v + s["res"].double() if case["residual"] else v


def _exact_product_train(s, case, seed):
    d = s["dout"].double()
    if case["act"]:
        v = s["pre"].double().requires_grad_()
        d, = torch.autograd.grad(_act64(v, case["act"]), v, d)
    return dict(dx=torch.mm(d, s["w"].double()), dw=torch.mm(d.T, s["x"].double()), db=d.sum(0) if case["bias"] else None)


def _factors64(case, x, gate, ig, A, gb, ib):
    """(decay, what a token adds) in 64 bits."""
    l = A * torch.sigmoid(gate + gb)
    u = x if ig is None else x * torch.sigmoid(ig + ib)
    return torch.exp(l), u * torch.sqrt(-torch.expm1(2 * l)) if case["normalize"] else u


def _inputs64(s):
    return [None if s[k] is None else s[k].double() for k in ("x", "gate", "ig", "A", "gb", "ib")]


def _exact_rec_step(s, case, seed):
    a, u = _factors64(case, *_inputs64(s))
    pool, rows = s["pool"].double(), s["index"].long()
    pool[rows] = a * pool[rows] + u
    return pool[rows], pool


def _exact_rec_prompt(s, case, seed):
    a, u = _factors64(case, *_inputs64(s))
    out, fin = torch.zeros_like(u), s["h0"].double()
    if not case["nseq"]:
        for t in range(case["seqlen"]):
            fin = a[:, t] * fin + u[:, t]
            out[:, t] = fin
        return out, fin
    for b, row in enumerate(_cuts(case, seed)):
        for q, t0, n in row:
            h = fin[q]
            for t in range(t0, t0 + n):
                h = a[b, t] * h + u[b, t]
                out[b, t] = h
            fin[q] = h
        h = torch.zeros_like(h)                                           # padding runs from a zero state
        for t in range(t0 + n, case["seqlen"]):
            h = a[b, t] * h + u[b, t]
            out[b, t] = h
    return out, fin


def _exact_rec_train(s, case, seed):
    names = [k for k in ("x", "gate", "ig", "A", "gb", "ib") if s[k] is not None]
    given = dict(zip(("x", "gate", "ig", "A", "gb", "ib"), _inputs64(s)))
    for k in names:
        given[k].requires_grad_()
    a, u = _factors64(case, *given.values())
    d, L = s["dout"].double(), case["seqlen"]
    with torch.no_grad():
        h, g, da = torch.zeros_like(u), torch.zeros_like(u), torch.zeros_like(u)
        h[:, 0] = u[:, 0]
        for t in range(1, L):
            h[:, t] = a[:, t] * h[:, t - 1] + u[:, t]
        g[:, L - 1] = d[:, L - 1]
        for t in reversed(range(L - 1)):
            g[:, t] = d[:, t] + a[:, t + 1] * g[:, t + 1]
        da[:, 1:] = g[:, 1:] * h[:, :-1]
    got = dict(zip(names, torch.autograd.grad((a, u), [given[k] for k in names], (da, g))))
    return dict(out=h, dx=got["x"], dgate=got["gate"], dA=got["A"], dig=got.get("ig"), dgb=got["gb"], dib=got.get("ib"))


EXACT = dict(norm=_exact_norm, norm_train=_exact_norm_train, norm_product8=_exact_norm_product8, product=_exact_product,
             product_train=_exact_product_train, rec_step=_exact_rec_step, rec_prompt=_exact_rec_prompt,
             rec_train=_exact_rec_train)


def work(case):
    """Bytes that have to move and operations that have to be done in one pass."""
    op, e = case["op"], ES[case["dtype"]]
    if op.startswith("norm"):
        M, K = case["rows"], case["width"]
        r = {"": 0, "same": e, "f32": 4}[case["residual"]]
        if op == "norm":
            return {"bytes": M * K * (2 * e + 2 * r) + 4 * K, "flops": 6 * M * K}
        if op == "norm_train":  # forward; the sum, dout (and the sum's gradient) -> dx (and dresidual, where its type is another)
            more = 2 * e + (e if not r else 2 * r + (e if r != e else 0))
            return {"bytes": M * K * (2 * e + 2 * r + more) + 12 * K, "flops": 18 * M * K}
        N = case["outs"]
        return {"bytes": M * K * (e + 2 * r) + N * K + M * N * e + 4 * (M + N + K), "flops": 2 * M * N * K}
    if op.startswith("product"):
        M, K, N = case["rows"], case["width"], case["outs"]
        if op == "product":
            return {"bytes": e * (M * K + N * K + M * N * (2 if case["residual"] else 1)) + (4 * N if case["bias"] else 0),
                    "flops": 2 * M * N * K}
        return {"bytes": e * (M * N * (2 if case["act"] else 1) + 2 * M * K + 2 * N * K) + (4 * N if case["bias"] else 0),
                "flops": 4 * M * N * K}
    Ch = case["channels"]
    tokens = case["batch"] * case.get("seqlen", 1)
    n, ins, par = tokens * Ch, 3 if case["in_gate"] else 2, 4 * Ch * (3 if case["in_gate"] else 2)
    if op == "rec_step":
        return {"bytes": n * (e * (ins + 1) + 2 * ES[case["state"]]) + par, "flops": 20 * n}
    if op == "rec_prompt":
        states = 2 * (case["nseq"] or case["batch"]) * Ch * ES[case["state"]]
        return {"bytes": n * e * (ins + 1) + par + states + (4 * tokens if case["nseq"] else 0), "flops": 20 * n}
    # forward: the inputs -> out; backward: the inputs and dout -> their gradients
    return {"bytes": n * e * (ins + 1 + 2 * ins + 1) + 3 * par, "flops": 60 * n}
