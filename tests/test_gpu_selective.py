"""GPU tests of the causal convolution, the selective scan and the 8-bit state cache against the 64-bit
loops of selective_ref.py.  Tolerances are the bounds derived there: half a step of the output's type plus
K u S, K the most roundings on a path from an input to the output:
  convolution: W + 2 in a sum, 40 for the gate;                 its dw, dbias: one more per token
  scan: 8 a token (step, exponential, two products, a sum), 2 N for the sums over n, 100 for softplus and gates;
        dB, dC: one more per channel of the group; dA, dD, ddt_bias: one more per token of the batch
"""
import pytest
import torch

import mamba_ssd_prefill_amd as ssd
import selective_ref as ref
from gpu_common import require_gpu, say

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def dev():
    return require_gpu()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def cuda(t):
    return None if t is None else t.cuda()


def packing(B, L, kind, g):
    """(seq_idx or None, number of states): runs of random lengths, numbers shuffled, padding at the end."""
    if kind is None:
        return None, B
    seq = torch.full((B, L), -1, dtype=torch.int32)
    cuts = []
    for b in range(B):
        used = L if kind == "full" else max(1, L - L // 5)
        if kind == "ones":
            at = list(range(used + 1))
        else:
            n = min(used, 4)
            at = [0] + sorted((torch.randperm(used - 1, generator=g)[:n - 1] + 1).tolist()) + [used]
        cuts += [(b, s, e) for s, e in zip(at, at[1:])]
    order = torch.randperm(len(cuts), generator=g).tolist()
    for q, (b, s, e) in zip(order, cuts):
        seq[b, s:e] = q
    return seq, len(cuts) + 1  # one number that no sequence uses


def strided(t, extra=6):
    """t as a view into rows that are `extra` elements longer."""
    row = t.flatten(2) if t.dim() > 2 else t
    wide = torch.full(row.shape[:-1] + (row.shape[-1] + extra,), float("nan"), dtype=t.dtype, device=t.device)
    wide[..., 2:2 + row.shape[-1]] = row
    return wide[..., 2:2 + row.shape[-1]].unflatten(-1, t.shape[2:]) if t.dim() > 3 else wide[..., 2:2 + row.shape[-1]]


# ---- convolution ---------------------------------------------------------------------------------------
CONV = [
    # (B, L, Ch, W, dtype, activation, packing, state, splits, strided)
    (1, 1, 1, 4, "f32", "silu", None, True, None, False),
    (2, 2, 5, 4, "bf16", None, None, True, None, False),
    (1, 3, 64, 4, "f16", "silu", None, False, None, False),
    (2, 77, 72, 4, "bf16", "silu", None, True, (40, 16, 16), False),
    (3, 50, 68, 3, "f16", "silu", "pad", True, (64, 4), True),
    (1, 130, 33, 2, "f32", None, "full", False, None, True),
    (2, 40, 24, 4, "f32", "silu", "ones", True, None, False),
    (1, 97, 128, 4, "bf16", "silu", "pad", True, None, False),
    (2, 16, 12, 3, "f32", "silu", "full", True, (5, 7), False),
]


def conv_case(case, seed):
    B, L, Ch, W, dtype, act, pack, state, splits, stride = case
    g, t = gen(seed), DT[dtype]
    seq, S = packing(B, L, pack, g)
    x, w, b = torch.randn(B, L, Ch, generator=g).to(t), 0.5 * torch.randn(Ch, W, generator=g), torch.randn(Ch, generator=g)
    h0 = torch.randn(S, Ch, W - 1, generator=g).to(t) if state else None
    xg = strided(x.cuda()) if stride else x.cuda()
    kw = dict(activation=act, seq_idx=cuda(seq), nseq=S if pack else None, initial_state=cuda(h0), splits=splits)
    return x, w, b, h0, seq, S, xg, kw, g


@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv(case):
    say("conv", case)
    B, L, Ch, W, dtype, act, pack, state, splits, _ = case
    x, w, b, h0, seq, S, xg, kw, _ = conv_case(case, 11)
    out, fin = ssd.causal_conv(xg, w.cuda(), b.cuda(), **kw)
    torch.cuda.synchronize()
    if splits:
        assert [o.shape[-1] for o in out] == list(splits) and all(o.is_contiguous() for o in out)
        out = torch.cat(out, -1)
    rr = ref.runs(B, L, seq)
    _, want, wfin = ref.conv(x, w, b, h0, S, act, rr)
    scale = ref.conv(x, w, b, h0, S, act, rr, absolute=True)[0]
    ref.close(out, want, scale, W + 42, x.dtype, "conv out")
    assert torch.equal(fin.cpu().double(), wfin)  # inputs as they were; zeros where no sequence is


@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv_backward(case):
    say("conv backward", case)
    B, L, Ch, W, dtype, act, pack, state, splits, _ = case
    x, w, b, h0, seq, S, xg, kw, g = conv_case(case, 12)
    dout = torch.randn(B, L, Ch, generator=g).to(x.dtype)
    dfin = torch.randn(S, Ch, W - 1, generator=g).to(x.dtype)
    dg = dout.cuda()
    if splits:
        dg = tuple(d.contiguous() for d in dg.split(splits, -1))
    runs = [ssd.causal_conv_backward(dg, xg, w.cuda(), b.cuda(), dfinal_state=dfin.cuda(), **kw) for _ in range(2)]
    torch.cuda.synchronize()
    got = runs[0]
    for p, q in zip(*runs):
        assert (p is None and q is None) or torch.equal(p, q)  # a fixed order of summation
    rr = ref.runs(B, L, seq)
    dout = used(dout, seq, S)
    want = ref.conv_grads(dout, dfin, x, w, b, h0, S, act, rr)
    scale = ref.conv_grads(dout, dfin, x, w, b, h0, S, act, rr, absolute=True)
    names, tokens = ("dx", "dw", "dbias", "dh0"), B * L
    for i, (a, t, k) in enumerate(zip(got, (x.dtype, torch.float32, torch.float32, x.dtype), (0, tokens, tokens, 0))):
        if a is not None:
            ref.close(a, want[i], scale[i], 2 * W + 60 + k, t, "conv " + names[i])
    assert (got.dinitial_state is None) == (h0 is None)


@pytest.mark.parametrize("dtype,W,Ch,B,slots", [("bf16", 4, 70, 5, 9), ("f32", 3, 64, 1, 1), ("f16", 2, 5, 3, 3)])
def test_conv_step_continues_the_prompt(dtype, W, Ch, B, slots):
    """A prompt of L0 tokens and then single tokens on a pool give the outputs of the whole prompt; a row without a
    slot touches nothing and gets zeros."""
    g, t = gen(13), DT[dtype]
    L, L0 = 12, 7
    x, w, b = torch.randn(B, L, Ch, generator=g).to(t).cuda(), torch.randn(Ch, W, generator=g).cuda(), torch.randn(Ch, generator=g).cuda()
    full, last = ssd.causal_conv(x, w, b)
    _, st = ssd.causal_conv(x[:, :L0].contiguous(), w, b)
    pool = torch.randn(slots, Ch, W - 1, generator=g).to(t).cuda()
    where = torch.randperm(slots, generator=g)[:B].to(torch.int32).cuda()
    pool[where.long()] = st
    before = pool.clone()
    for k in range(L0, L):
        xk = torch.cat([x[:, k], x[:1, k]])            # one padded row more
        sl = torch.cat([where, torch.tensor([-1 if k % 2 else slots], dtype=torch.int32, device="cuda")])
        out = ssd.causal_conv_step(xk, w, b, state=pool, slots=sl)
        torch.cuda.synchronize()
        assert torch.equal(out[:B], full[:, k]) and not out[B].any()
    assert torch.equal(pool[where.long()], last)
    rest = torch.ones(slots, dtype=torch.bool)
    rest[where.long().cpu()] = False
    assert torch.equal(pool[rest.cuda()], before[rest.cuda()])
    # without slots, and split
    own = st.clone()
    o = ssd.causal_conv_step(x[:, L0], w, b, state=own, splits=(2, 1, Ch - 3), activation=None)
    assert [v.shape[-1] for v in o] == [2, 1, Ch - 3]
    want = ssd.causal_conv(x[:, L0:L0 + 1].contiguous(), w, b, activation=None, initial_state=st)[0][:, 0]
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(o, -1), want)


# ---- scan ------------------------------------------------------------------------------------------------
SCAN = [
    # (B, L, D, N, G, dtype, state dtype, packing, state, gate, D and bias, softplus, strided)
    (1, 1, 1, 8, 1, "f32", "f32", None, True, True, True, True, False),
    (2, 17, 65, 16, 1, "bf16", "f32", None, True, True, True, True, False),
    (1, 16, 64, 16, 1, "f16", "f16", None, False, False, False, True, False),
    (3, 40, 90, 16, 3, "bf16", "bf16", None, True, True, True, True, True),
    (2, 33, 130, 32, 2, "f32", "f32", "pad", True, True, True, True, True),
    (1, 100, 63, 64, 1, "f16", "f32", "pad", True, True, True, True, False),
    (2, 21, 8, 8, 4, "bf16", "f32", "ones", True, False, True, True, False),
    (1, 75, 70, 16, 1, "f32", "f32", "full", False, True, False, False, True),
    (1, 5, 128, 64, 2, "bf16", "f32", None, True, True, True, True, True),
]


def scan_inputs(B, L, D, N, G, dtype, sdtype, pack, state, gate, params, softplus, seed):
    g, t = gen(seed), DT[dtype]
    seq, S = packing(B, L, pack, g)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    # steps of 0.02 .. 1 and decays of -0.5 .. -N / 4: memories from a token to dozens
    raw = rn(B, L, D) - 1.5
    s = dict(x=rn(B, L, D).to(t), dt=(raw if softplus else 0.02 + 0.3 * raw.abs()).to(t),
             A=-(0.5 + torch.rand(D, N, generator=g) * N / 4), B=rn(B, L, G, N).to(t), C=rn(B, L, G, N).to(t),
             D=rn(D) if params else None, bias=0.3 * rn(D) if params and softplus else None,
             z=rn(B, L, D).to(t) if gate else None, h0=rn(S, D, N).to(DT[sdtype]) if state else None)
    return s, seq, S, g


def call_args(s, stride=False):
    v = {k: cuda(t) for k, t in s.items()}
    if stride:
        for k in ("x", "dt", "z", "B", "C"):
            if v[k] is not None:
                v[k] = strided(v[k])
    return (v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["bias"], v["z"]), v["h0"]


def ref_args(s):
    return s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["bias"], s["z"], s["h0"]


def check_scan(got, s, S, softplus, rr, L, N, sdtype, name):
    want, wfin, _, _ = ref.scan(*ref_args(s), S, softplus, rr)
    scale, sfin, _, _ = ref.scan(*ref_args(s), S, softplus, rr, absolute=True)
    K = 8 * L + 2 * N + 100
    ref.close(got[0], want, scale, K, s["x"].dtype, name + " out")
    if got[1] is not None:
        ref.close(got[1], wfin, sfin, K, DT[sdtype], name + " state")


@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan(case):
    say("scan", case)
    B, L, D, N, G, dtype, sdtype, pack, state, gate, params, softplus, stride = case
    s, seq, S, _ = scan_inputs(*case[:-1], seed=21)
    args, h0 = call_args(s, stride)
    got = ssd.selective_scan(*args, dt_softplus=softplus, seq_idx=cuda(seq), nseq=S if pack else None, initial_state=h0,
                             state_dtype=DT[sdtype])
    torch.cuda.synchronize()
    check_scan(got, s, S, softplus, ref.runs(B, L, seq), L, N, sdtype, "scan")


@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan_backward(case):
    say("scan backward", case)
    B, L, D, N, G, dtype, sdtype, pack, state, gate, params, softplus, stride = case
    s, seq, S, g = scan_inputs(*case[:-1], seed=22)
    args, h0 = call_args(s, stride)
    kw = dict(dt_softplus=softplus, seq_idx=cuda(seq), nseq=S if pack else None, initial_state=h0, state_dtype=DT[sdtype])
    out, fin, saved = ssd.selective_scan(*args, save_for_backward=True, **kw)
    plain = ssd.selective_scan(*args, **kw)
    assert torch.equal(out, plain[0]) and torch.equal(fin, plain[1])
    dout = torch.randn(B, L, D, generator=g).to(s["x"].dtype)
    dfin = torch.randn(S, D, N, generator=g).to(DT[sdtype])
    two = [ssd.selective_scan_backward(dout.cuda(), *args, saved=saved, dfinal_state=dfin.cuda(), **kw) for _ in range(2)]
    torch.cuda.synchronize()
    for p, q in zip(*two):
        assert (p is None and q is None) or torch.equal(p, q)  # a fixed order of summation
    check_grads(two[0], used(dout, seq, S), dfin, s, S, softplus, ref.runs(B, L, seq), case)


def used(dout, seq, S):
    """The output gradients that count: none at padded tokens."""
    return dout if seq is None else dout * ((seq >= 0) & (seq < S))[..., None]


def check_grads(got, dout, dfin, s, S, softplus, rr, case):
    B, L, D, N, G, dtype, sdtype = case[:7]
    want = ref.scan_grads(dout, dfin, *ref_args(s), S, softplus, rr)
    scale = ref.scan_grads(dout, dfin, *ref_args(s), S, softplus, rr, absolute=True)
    K, t = 8 * L + 2 * N + 100, s["x"].dtype
    for name, a, typ, more in (("dx", got.dx, t, 0), ("ddt", got.ddt, t, 0), ("dB", got.dB, t, D // G),
                               ("dC", got.dC, t, D // G), ("dz", got.dz, t, 0), ("dA", got.dA, torch.float32, B * L),
                               ("dD", got.dD, torch.float32, B * L), ("dbias", got.ddt_bias, torch.float32, B * L),
                               ("dh0", got.dinitial_state, DT[sdtype], 0)):
        if a is not None:
            ref.close(a, want[name], scale[name], K + more, typ, name)
    for a, k in ((got.dz, "z"), (got.dD, "D"), (got.ddt_bias, "bias"), (got.dinitial_state, "h0")):
        assert (a is None) == (s[k] is None)


LONG = [
    # long axes: (B, L, D, N, G, dtype, state dtype, packing, state, gate, D and bias, softplus)
    (1, 1000, 20, 16, 1, "f32", "f32", None, True, True, True, True),
    (1, 1601, 20, 8, 2, "bf16", "f32", "pad", True, True, True, True),
    (2, 700, 10, 64, 1, "f16", "f32", "full", True, False, True, True),
    (1, 513, 70, 32, 1, "f32", "f32", None, False, True, True, True),
]


@pytest.mark.parametrize("case", LONG, ids=str)
def test_scan_long(case):
    say("scan long", case)
    B, L, D, N, G, dtype, sdtype, pack, state, gate, params, softplus = case
    s, seq, S, g = scan_inputs(*case, seed=23)
    args, h0 = call_args(s)
    kw = dict(seq_idx=cuda(seq), nseq=S if pack else None, initial_state=h0, state_dtype=DT[sdtype])
    out, fin, saved = ssd.selective_scan(*args, save_for_backward=True, **kw)
    dout, dfin = torch.randn(B, L, D, generator=g).to(s["x"].dtype), torch.randn(S, D, N, generator=g).to(DT[sdtype])
    grads = ssd.selective_scan_backward(dout.cuda(), *args, saved=saved, dfinal_state=dfin.cuda(), **kw)
    torch.cuda.synchronize()
    rr = ref.runs(B, L, seq)
    # memories end after a few hundred tokens (decays of at least exp(-0.5 * 0.02) a token, sums of positive
    # scales), so a path has no more roundings that matter than one of 400 tokens; dA's sums run over all
    check_scan((out, fin), s, S, softplus, rr, min(L, 400), N, sdtype, "long")
    check_grads(grads, used(dout, seq, S), dfin, s, S, softplus, rr, (B, L) + case[2:])


def test_scan_of_a_prompt_in_two_calls_and_steps():
    """A prompt, its two halves with the state handed on, and its last tokens one by one on a pool."""
    B, L, D, N = 3, 60, 100, 16
    s, _, _, _ = scan_inputs(B, L, D, N, 1, "f32", "f32", None, True, True, True, True, seed=24)
    (x, dt, A, Bm, C, Dp, bias, z), h0 = call_args(s)
    full, fin = ssd.selective_scan(x, dt, A, Bm, C, Dp, bias, z, initial_state=h0)
    cut = lambda t, a, b: t[:, a:b]  # noqa: E731  (rows a constant distance apart only within one batch row)
    halves, st = [], h0
    for a, b in ((0, 29), (29, 50)):
        o, st = ssd.selective_scan(*[cut(t, a, b).contiguous() for t in (x, dt)], A, *[cut(t, a, b).contiguous() for t in (Bm, C)],
                                   Dp, bias, cut(z, a, b).contiguous(), initial_state=st)
        halves.append(o)
    pool = torch.full((B + 3, D, N), 7.0, device="cuda")
    where = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool[where.long()] = st
    slots = torch.cat([where, torch.tensor([-5], dtype=torch.int32, device="cuda")])
    pad = lambda t: torch.cat([t, t[:1]])  # noqa: E731
    for t in range(50, L):
        o = ssd.selective_scan_step(pad(x[:, t]), pad(dt[:, t]), A, pad(Bm[:, t]), pad(C[:, t]), Dp, bias, pad(z[:, t]),
                                    state=pool, slots=slots)
        torch.cuda.synchronize()
        assert not o[B].any()
        halves.append(o[:B, None])
    got = torch.cat(halves, 1)
    rr = ref.runs(B, L)
    scale, sfin, _, _ = ref.scan(*ref_args(s), B, True, rr, absolute=True)
    # both sides within K u S of the exact result
    for a, b, sc in ((got, full, scale), (pool[where.long()], fin, sfin)):
        assert bool(((a - b).double().abs().cpu() <= 2 * (8 * L + 2 * N + 100) * ref.U * sc + 1e-30).all())
    assert bool((pool[[1, 3, 5]] == 7.0).all())


@pytest.mark.parametrize("dtype,sdtype,N,D,G,B", [("bf16", "f32", 16, 100, 1, 4), ("f16", "f16", 64, 33, 3, 2),
                                                  ("f32", "bf16", 8, 7, 1, 1), ("bf16", "f32", 32, 256, 2, 9)])
def test_scan_step(dtype, sdtype, N, D, G, B):
    s, _, _, _ = scan_inputs(B, 1, D, N, G, dtype, sdtype, None, True, True, True, True, seed=25)
    (x, dt, A, Bm, C, Dp, bias, z), h0 = call_args(s)
    st = h0.clone()
    out = ssd.selective_scan_step(x[:, 0], dt[:, 0], A, Bm[:, 0], C[:, 0], Dp, bias, z[:, 0], state=st)
    torch.cuda.synchronize()
    check_scan((out[:, None], st), s, B, True, ref.runs(B, 1), 1, N, sdtype, "step")


def test_scan_gradients_against_differences():
    """The change of sum(out * w) + sum(final state * v) along random directions of all inputs, by central
    differences of the 64-bit loops, against the kernel's gradients in fp32."""
    B, L, D, N, G = 2, 23, 12, 16, 2
    s, seq, S, g = scan_inputs(B, L, D, N, G, "f32", "f32", "pad", True, True, True, True, seed=26)
    rr = ref.runs(B, L, seq)
    args, h0 = call_args(s)
    kw = dict(seq_idx=seq.cuda(), nseq=S, initial_state=h0)
    w, v = used(torch.randn(B, L, D, generator=g), seq, S), torch.randn(S, D, N, generator=g)
    _, _, saved = ssd.selective_scan(*args, save_for_backward=True, **kw)
    grads = ssd.selective_scan_backward(w.cuda(), *args, saved=saved, dfinal_state=v.cuda(), **kw)
    by = dict(x=grads.dx, dt=grads.ddt, A=grads.dA, B=grads.dB, C=grads.dC, D=grads.dD, bias=grads.ddt_bias, z=grads.dz,
              h0=grads.dinitial_state)

    def value(p):
        out, fin, _, _ = ref.scan(*ref_args(p), S, True, rr)
        return float((out * w.double()).sum() + (fin * v.double()).sum())
    for k in by:
        d = torch.randn(s[k].shape, generator=g).double()
        eps = 1e-5
        hi, lo = dict(s), dict(s)
        hi[k], lo[k] = s[k].double() + eps * d, s[k].double() - eps * d
        slope = (value(hi) - value(lo)) / (2 * eps)
        got = float((by[k].cpu().double() * d).sum())
        # the difference is right to eps^2; the gradient to (8 L + 2 N + 100) u of its absolute sum
        assert abs(got - slope) <= 5e-5 * float((by[k].cpu().double() * d).abs().sum()) + 1e-6, (k, got, slope)


def test_scan_values_at_the_edges():
    """Large steps and decays (the decay underflows to 0), zero steps (the state stays), a zero decay."""
    B, L, D, N = 1, 20, 64, 16
    s, _, _, _ = scan_inputs(B, L, D, N, 1, "f32", "f32", None, True, False, False, False, seed=27)
    s["dt"][:, 5] = 0.0
    s["dt"][:, 7] = 1000.0
    s["A"][3] = 0.0
    args, h0 = call_args(s)
    got = ssd.selective_scan(*args, dt_softplus=False, initial_state=h0)
    torch.cuda.synchronize()
    assert torch.isfinite(got[0]).all()
    check_scan(got, s, B, False, ref.runs(B, L), L, N, "f32", "edges")


def test_scan_softplus_of_small_and_large_arguments():
    """softplus over its whole range, seen through out = d x B C with one token: right to 100 u."""
    D, N = 4096, 8
    v = torch.linspace(-40, 40, D)
    s = dict(x=torch.ones(1, 1, D), dt=v.view(1, 1, D).clone(), A=-torch.ones(D, N), B=torch.ones(1, 1, 1, N),
             C=torch.zeros(1, 1, 1, N), D=None, bias=None, z=None, h0=None)
    s["C"][..., 0] = 1
    args, _ = call_args(s)
    out, _ = ssd.selective_scan(*args)
    want = torch.logaddexp(v.double(), torch.zeros((), dtype=torch.float64))
    assert float(((out.view(-1).cpu().double() - want).abs() / want).max()) <= 100 * ref.U


def test_padding_and_other_sequences_do_not_leak():
    """NaN in padded tokens and in another sequence reaches neither the outputs nor the gradients of the rest."""
    B, L, D, N = 1, 50, 64, 16
    s, _, _, g = scan_inputs(B, L, D, N, 1, "bf16", "f32", None, False, True, True, True, seed=28)
    seq = torch.tensor([[0] * 21 + [1] * 13 + [-1] * 16], dtype=torch.int32)
    bad = {k: (None if t is None else t.clone()) for k, t in s.items()}
    for k in ("x", "dt", "B", "C", "z"):
        bad[k][:, 34:] = float("nan")
    dout = torch.randn(B, L, D, generator=g).bfloat16()
    res = []
    for inp in (s, bad):
        args, _ = call_args(inp)
        kw = dict(seq_idx=seq.cuda(), nseq=2)
        out, fin, saved = ssd.selective_scan(*args, save_for_backward=True, **kw)
        gr = ssd.selective_scan_backward(dout.cuda(), *args, saved=saved, **kw)
        cx, cfin = ssd.causal_conv(args[0], torch.ones(D, 4, device="cuda"), seq_idx=kw["seq_idx"], nseq=2)
        res.append([t[:, :34] for t in (out, gr.dx, gr.ddt, gr.dB, gr.dC, gr.dz, cx)] + [fin, cfin])
    torch.cuda.synchronize()
    for a, b in zip(*res):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


# ---- cache -------------------------------------------------------------------------------------------------
def same(a, b):
    """Equal values, a NaN equal to a NaN (the scale and the values of a group that holds an infinity)."""
    return a.dtype == b.dtype and a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("shape,group,fmt,dtype,B,slots", [
    ((4, 64, 128), 128, "int8", "f32", 3, 5), ((7, 16), 16, "e4m3", "f16", 2, 2), ((130, 32), 64, "e4m3", "f32", 4, 9),
    ((3, 16, 64), 32, "int8", "bf16", 1, 3), ((5120, 16), 16, "int8", "f16", 2, 2), ((1, 16), 16, "e4m3", "bf16", 3, 4)])
def test_cache_round_trip(shape, group, fmt, dtype, B, slots):
    g, t = gen(31), DT[dtype]
    v = (torch.randn(B, *shape, generator=g) * torch.exp(3 * torch.randn(B, shape[0], *[1] * (len(shape) - 1), generator=g))).to(t)
    flat = v.view(B, -1)
    flat[0, :group] = 0                                                    # a group of zeros
    if dtype == "f32":
        flat[-1, :group] = torch.arange(group).float() - group / 2         # quotients on borders
        flat[-1, 0] = 127.0 if fmt == "int8" else 448.0                    # scale 1
        flat[-1, 1:9] = torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, 17.0, 0.0009765625, 0.0029296875])
    codes, scales = ssd.state_cache(slots, shape, group=group, format=fmt)
    where = torch.randperm(slots, generator=g)[:B].to(torch.int32).cuda()
    ssd.state_cache_write(v.cuda(), codes, scales, where)
    back = ssd.state_cache_read(codes, scales, where, state_dtype=t)
    torch.cuda.synchronize()
    want, ws = ref.cache(v, group, fmt)
    assert same(scales[where.long()].cpu().double(), ws)
    assert same(back.cpu(), want.float().to(t))                    # one product in fp32, then the type
    held = codes[where.long()].float() * scales[where.long()].view(B, -1, 1).expand(B, -1, group).reshape(B, *shape)
    assert same(held.to(t), back)                                  # the codes are the type's own values
    rest = torch.ones(slots, dtype=torch.bool)
    rest[where.long().cpu()] = False
    assert not codes.view(torch.int8)[rest.cuda()].any() and not scales[rest.cuda()].any()
    # without slots: every slot in order
    whole = ssd.state_cache_read(codes, scales)
    assert whole.dtype == torch.float32 and same(whole[where.long()].to(t), back)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_cache_borders_between_codes(fmt):
    """Quotients at and next to every border between two codes round as the exact quotient does."""
    most = 127.0 if fmt == "int8" else 448.0
    if fmt == "int8":
        border = torch.arange(0, 127).float() + 0.5
    else:
        vals = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
        border = (vals[1:] + vals[:-1]) / 2
    rows = []
    for s in (1.0, 3.0, 0.1, 1.7e-7, 12345.678):
        s = torch.tensor(s)
        top = (most * s.double()).float()
        scale = (top.double() / most).float().double()
        mid = (border.double() * scale).float()
        for d in (0.0, float("inf"), float("-inf")):
            m = mid if d == 0.0 else torch.nextafter(mid, torch.full_like(mid, d))
            for part in m.split(63):
                row = torch.zeros(64)
                row[0], row[1:1 + len(part)] = top, part
                rows.append(row)
    v = torch.stack(rows + [-r for r in rows])
    codes, scales = ssd.state_cache(len(v), (64,), group=64, format=fmt)
    ssd.state_cache_write(v.cuda(), codes, scales)
    torch.cuda.synchronize()
    want, ws = ref.cache(v, 64, fmt)
    assert torch.equal(ssd.state_cache_read(codes, scales).cpu(), want.float())


def test_cache_special_values():
    v = torch.randn(6, 64, generator=gen(32))
    v[0, 3] = float("inf")
    v[1, 40] = float("nan")
    v[2] = 1e-38            # below the smallest scale
    v[3, 5] = 3.4e38        # the largest
    v[4] = 0
    codes, scales = ssd.state_cache(6, (64,), group=32)
    slots = torch.tensor([0, 1, 2, 3, 4, 6], dtype=torch.int32, device="cuda")  # the last has no slot
    scales[5] = 2.0
    ssd.state_cache_write(v.cuda(), codes, scales, slots)
    back = ssd.state_cache_read(codes, scales, slots, out=torch.full((6, 64), 9.0, device="cuda")).cpu()
    torch.cuda.synchronize()
    assert back[0, :32].isnan().all() and torch.isfinite(back[0, 32:]).all()
    assert back[1, 32:].isnan().all() and torch.isfinite(back[1, :32]).all()
    assert not back[2].any() and not back[4].any() and not back[5].any()
    assert abs(back[3, 5] / 3.4e38 - 1) < 0.01
    assert bool((scales[5] == 2.0).all()) and not codes[5].any()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_cache_quotients_below_the_fp32_range(fmt):
    """Values so far below their group's largest that their quotient leaves fp32, of either sign, are code 0."""
    v = torch.zeros(2, 32)
    v[:, 0] = torch.tensor([1e30, 3e38])
    v[:, 1:9] = torch.tensor([1e-45, -1e-45, 1e-38, -1e-38, 3e-39, -3e-39, 1e-20, -1e-20])
    codes, scales = ssd.state_cache(2, (32,), group=16, format=fmt)
    ssd.state_cache_write(v.cuda(), codes, scales)
    back = ssd.state_cache_read(codes, scales).cpu()
    torch.cuda.synchronize()
    assert not back[:, 1:].any() and torch.equal(back, ref.cache(v, 16, fmt)[0].float())


# ---- together ------------------------------------------------------------------------------------------------
def layer(p, u, state=None, pos=None):
    """One selective layer's inner path on raw activations u = [x | z], as a model holds it: a joint projection's
    halves as views, the convolution, then the scan."""
    D = p["A"].shape[0]
    x, z = u[..., :D], u[..., D:]
    xc, cs = ssd.causal_conv(x, p["w"], p["b"], initial_state=None if state is None else state[0])
    dbc = xc @ p["proj"]
    R, N = p["R"], p["A"].shape[1]
    dt = dbc[..., :R] @ p["dtp"]
    B, C = dbc[..., R:R + N].unsqueeze(-2), dbc[..., R + N:].unsqueeze(-2)
    out, hs = ssd.selective_scan(xc, dt, p["A"], B, C, p["D"], p["bias"], z, initial_state=None if state is None else state[1])
    return out, (cs, hs)


def layer_params(D, N, R, t):
    g = gen(41)
    return dict(w=0.5 * torch.randn(D, 4, generator=g).cuda(), b=0.1 * torch.randn(D, generator=g).cuda(), R=R,
                proj=(torch.randn(D, R + 2 * N, generator=g) / D ** 0.5).to(t).cuda(),
                dtp=(torch.randn(R, D, generator=g) / R ** 0.5).to(t).cuda(), A=-(1 + torch.rand(D, N, generator=g) * N).cuda(),
                D=torch.randn(D, generator=g).cuda(), bias=(torch.randn(D, generator=g) - 3).cuda())


def test_prompt_cache_and_steps_together():
    """Two prompts through convolution and scan, their scan states into the 8-bit pool and back, and three
    tokens more on pools: the tokens' outputs are those of the whole prompts, up to the error that the
    8-bit state brings in (at most half a code of each group's largest value, through C and the gate)."""
    B, L, D, N, R = 2, 45, 96, 16, 6
    p = layer_params(D, N, R, torch.float32)
    u = torch.randn(B, L + 3, 2 * D, generator=gen(42)).cuda()
    full, _ = layer(p, u)
    first, (cs, hs) = layer(p, u[:, :L].contiguous())
    codes, scales = ssd.state_cache(4, (D, N), group=16)
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    ssd.state_cache_write(hs, codes, scales, slots)
    exact_pool, pool, conv_pool = (torch.zeros(4, *s.shape[1:], dtype=s.dtype, device="cuda") for s in (hs, hs, cs))
    back = ssd.state_cache_read(codes, scales, slots)
    pool[slots.long()], exact_pool[slots.long()], conv_pool[slots.long()] = back, hs, cs
    half = scales[slots.long()] / 2
    assert bool(((back - hs).abs() <= half[..., None].expand(-1, -1, 16).reshape(hs.shape) * (1 + 1e-6)).all())
    for t in range(L, L + 3):
        xc = ssd.causal_conv_step(u[:, t, :D], p["w"], p["b"], state=conv_pool, slots=slots)
        dbc = xc @ p["proj"]
        dt, Bt, Ct = dbc[:, :R] @ p["dtp"], dbc[:, None, R:R + N], dbc[:, None, R + N:]
        a = ssd.selective_scan_step(xc, dt, p["A"], Bt, Ct, p["D"], p["bias"], u[:, t, D:], state=exact_pool, slots=slots)
        b = ssd.selective_scan_step(xc, dt, p["A"], Bt, Ct, p["D"], p["bias"], u[:, t, D:], state=pool, slots=slots)
        # torch's products on one row and on a prompt sum in other orders, in fp32: D terms of size 1 / D^0.5
        assert bool((a - full[:, t]).abs().max() <= 1e-4 * (1 + full[:, t].abs().max()))
        z = u[:, t, D:]
        gate = (z * torch.sigmoid(z)).abs()
        reach = (Ct.abs() * half[..., None].expand(-1, -1, 16).reshape(hs.shape)).sum(-1) * gate  # decays are at most 1
        assert bool(((a - b).abs() <= reach * 1.001 + 1e-5).all())


def test_mamba2_block_by_single_tokens():
    """The short convolution's step, split into x, B and C, feeds ssd_decode_step: a Mamba-2 block's tokens one by
    one equal its prompt (conv_silu and ssd_prefill)."""
    B, L, H, P, G, N = 2, 9, 4, 64, 1, 64
    g, t = gen(43), torch.bfloat16
    Ch = H * P + 2 * G * N
    xbc = torch.randn(B, L, Ch, generator=g).to(t).cuda()
    w, b = 0.5 * torch.randn(Ch, 4, generator=g).cuda(), 0.1 * torch.randn(Ch, generator=g).cuda()
    dt = torch.randn(B, L, H, generator=g).to(t).cuda()
    A, D, bias = (-torch.rand(H, generator=g) - 0.5).cuda(), torch.randn(H, generator=g).cuda(), (torch.randn(H, generator=g) - 2).cuda()
    x, Bm, Cm = ssd.conv_silu(xbc, w, b, nheads=H, headdim=P, ngroups=G, dstate=N)
    y, fin = ssd.ssd_prefill(x, dt, A, Bm, Cm, D, bias)
    (x2, B2, C2), cs = ssd.causal_conv(xbc, w, b, splits=(H * P, G * N, G * N))
    assert torch.equal(x2.view_as(x), x) and torch.equal(B2.view_as(Bm), Bm) and torch.equal(C2.view_as(Cm), Cm)
    cpool, state = torch.zeros(B, Ch, 3, dtype=t, device="cuda"), torch.zeros(B, H, P, N, device="cuda")
    for k in range(L):
        xt, Bt, Ct = ssd.causal_conv_step(xbc[:, k], w, b, state=cpool, splits=(H * P, G * N, G * N))
        assert torch.equal(xt, x2[:, k]) and torch.equal(Bt, B2[:, k]) and torch.equal(Ct, C2[:, k])
        yt, state = ssd.ssd_decode_step(xt.view(B, H, P), dt[:, k].contiguous(), A, Bt.view(B, G, N), Ct.view(B, G, N), D, bias,
                                        state)
        torch.cuda.synchronize()
        # each side rounds once to bf16, and the prefill's products round their operands to it
        assert bool((yt.float() - y[:, k].float()).abs().max() <= 0.05 * y[:, k].float().abs().max())
    assert torch.equal(cpool, cs)
    assert bool((state - fin).abs().max() <= 0.02 * fin.abs().max())


def test_captured_and_replayed():
    """Prompt, backward, steps and cache in one HIP graph, replayed with other inputs between eager calls: every
    replay equals the eager result on the same inputs."""
    B, L, D, N = 2, 37, 130, 16
    s, _, _, g = scan_inputs(B, L, D, N, 1, "bf16", "f32", None, True, True, True, True, seed=29)
    (x, dt, A, Bm, C, Dp, bias, z), h0 = call_args(s)
    w, dout = torch.randn(D, 4, generator=g).cuda(), torch.randn(B, L, D, generator=g).bfloat16().cuda()
    start = torch.randn(3, D, N, generator=g).cuda()
    pool = start.clone()
    codes, scales = ssd.state_cache(3, (D, N), group=16)

    def work():
        pool.copy_(start)
        xc, cs = ssd.causal_conv(x, w)
        out, fin, saved = ssd.selective_scan(xc, dt, A, Bm, C, Dp, bias, z, initial_state=h0, save_for_backward=True)
        gr = ssd.selective_scan_backward(dout, xc, dt, A, Bm, C, Dp, bias, z, saved=saved, initial_state=h0)
        cg = ssd.causal_conv_backward(gr.dx, x, w)
        o = ssd.selective_scan_step(xc[:, -1], dt[:, -1], A, Bm[:, -1], C[:, -1], Dp, bias, z[:, -1], state=pool,
                                    slots=torch_slots)
        ssd.state_cache_write(fin, codes, scales, torch_slots)
        return [out, fin, *gr, cg.dx, cg.dweight, o, pool, cs, ssd.state_cache_read(codes, scales, torch_slots)]
    torch_slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for k in range(3):
        x.copy_(torch.randn(B, L, D, generator=g).to(x.dtype))
        dout.copy_(torch.randn(B, L, D, generator=g).to(x.dtype))
        graph.replay()
        torch.cuda.synchronize()
        got = [None if t is None else t.clone() for t in held]
        want = [None if t is None else t.clone() for t in work()]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert (a is None and b is None) or torch.equal(a, b)


def test_two_streams_at_once():
    """Calls in flight on two streams (their own workspaces) give what they give alone."""
    s, _, _, _ = scan_inputs(1, 600, 64, 16, 1, "bf16", "f32", None, True, True, True, True, seed=30)
    args, h0 = call_args(s)
    want = ssd.selective_scan(*args, initial_state=h0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for st in streams * 2:
        with torch.cuda.stream(st):
            got.append(ssd.selective_scan(*args, initial_state=h0))
    torch.cuda.synchronize()
    for o, f in got:
        assert torch.equal(o, want[0]) and torch.equal(f, want[1])


def test_refusals_on_the_gpu():
    """Shapes the library does not take come back as errors and leave the device usable."""
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    for bad in (lambda: ssd.selective_scan(z(1, 4, 8), z(1, 4, 8), z(8, 24), z(1, 4, 1, 24), z(1, 4, 1, 24)),
                lambda: ssd.selective_scan(z(1, 0, 8), z(1, 0, 8), z(8, 16), z(1, 0, 1, 16), z(1, 0, 1, 16)),
                lambda: ssd.selective_scan(z(1, 4, 9), z(1, 4, 9), z(9, 16), z(1, 4, 2, 16), z(1, 4, 2, 16)),
                lambda: ssd.causal_conv(z(1, 4, 8), z(8, 5)), lambda: ssd.causal_conv(z(0, 4, 8), z(8, 4))):
        with pytest.raises(ssd.SSDError):
            bad()
    x = z(1, 4, 8)
    st = z(1, 8, 16)
    for bad in (lambda: ssd.selective_scan(x, x, z(8, 16), z(1, 4, 1, 16), z(1, 4, 1, 16), initial_state=st, final_state=st),
                lambda: ssd.selective_scan(x, x, z(8, 16), z(1, 4, 1, 16), z(1, 4, 1, 16), workspace=z(1, t=torch.uint8))):
        with pytest.raises(ssd.SSDError):
            bad()
    with pytest.raises(ValueError):
        ssd.selective_scan(x, x.half(), z(8, 16), z(1, 4, 1, 16), z(1, 4, 1, 16))
    with pytest.raises(ValueError):
        ssd.selective_scan(x, x.cpu(), z(8, 16), z(1, 4, 1, 16), z(1, 4, 1, 16))
    out, _ = ssd.causal_conv(x + 1, torch.ones(8, 4, device="cuda"), activation=None)
    assert out[0, :, 0].tolist() == [1, 2, 3, 4]


def test_growing_states_over_splits():
    """Negative steps grow the state; a zero state stays zero over a split whose decays' product overflows."""
    L, D, N = 4096, 64, 16
    x = torch.zeros(1, L, D, device="cuda")
    x[:, -1] = 1
    dt = torch.full((1, L, D), -1.0, device="cuda")
    A = -torch.ones(D, N, device="cuda")
    B = torch.ones(1, L, 1, N, device="cuda")
    out, fin, saved = ssd.selective_scan(x, dt, A, B, B, dt_softplus=False, save_for_backward=True)
    g = ssd.selective_scan_backward(x, x, dt, A, B, B, saved=saved, dt_softplus=False)
    torch.cuda.synchronize()
    assert not out[:, :-1].any() and bool((out[:, -1] == -N).all()) and bool((fin == -1).all())
    assert bool((g.dC[0, -1] == -D).all()) and bool((g.dx[0, -1] == -N).all())


def test_given_outputs_and_workspaces():
    """Outputs and workspaces handed in are used, and states of numbers that no sequence uses stay as they were."""
    s, seq, S, g = scan_inputs(2, 30, 70, 16, 1, "bf16", "f32", "pad", True, True, True, True, seed=51)
    args, h0 = call_args(s)
    kw = dict(seq_idx=seq.cuda(), nseq=S, initial_state=h0)
    want, wfin = ssd.selective_scan(*args, **kw)
    out, fin = torch.full_like(want, 5.0), torch.full_like(wfin, 5.0)
    space = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    o, f = ssd.selective_scan(*args, out=out, final_state=fin, workspace=space, **kw)
    cfin = torch.full((S, 70, 3), 5.0, dtype=torch.bfloat16, device="cuda")
    cw, cb = torch.randn(70, 4, generator=g).cuda(), torch.randn(70, generator=g).cuda()
    _, cf = ssd.causal_conv(args[0], cw, cb, seq_idx=kw["seq_idx"], nseq=S, final_state=cfin)
    gr = [ssd.causal_conv_backward(want, args[0], cw, cb, seq_idx=kw["seq_idx"], nseq=S, workspace=w) for w in (None, space)]
    torch.cuda.synchronize()
    assert o.data_ptr() == out.data_ptr() and f.data_ptr() == fin.data_ptr() and cf.data_ptr() == cfin.data_ptr()
    assert torch.equal(o, want) and torch.equal(f[:-1], wfin[:-1]) and bool((f[-1] == 5.0).all())
    assert bool((cf[-1] == 5.0).all()) and not bool((cf[:-1] == 5.0).all())
    assert all(torch.equal(a, b) for a, b in zip(*gr) if a is not None)
    with pytest.raises(ssd.SSDError):
        ssd.selective_scan_backward(want, *args, saved=ssd.selective_scan(*args, save_for_backward=True, **kw)[2],
                                    workspace=space[:256], **kw)


def test_offsets_past_32_bits():
    """Rows, pools and caches whose offsets pass 2^32 bytes (and 2^31 elements)."""
    g = gen(52)
    D, N, L = 64, 16, 300
    row = 1 << 23                                                          # elements between rows: 5 GB in all
    wide = torch.empty(L, row, dtype=torch.bfloat16, device="cuda")
    x, dt, B, C = (torch.randn(1, L, n, generator=g).bfloat16().cuda() for n in (D, D, N, N))
    far = []
    for i, t in enumerate((x, dt, B, C)):
        v = wide.unsqueeze(0)[..., 128 * i:128 * i + t.shape[-1]]
        v.copy_(t)
        far.append(v)
    A, w = -torch.rand(D, N, generator=g).cuda() - 0.1, torch.randn(D, 4, generator=g).cuda()
    near = ssd.selective_scan(x, dt, A, B.unsqueeze(2), C.unsqueeze(2), save_for_backward=True)
    got = ssd.selective_scan(far[0], far[1], A, far[2].unsqueeze(2), far[3].unsqueeze(2), save_for_backward=True)
    for a, b in zip(near, got):
        assert torch.equal(a, b)
    ga = ssd.selective_scan_backward(x, x, dt, A, B.unsqueeze(2), C.unsqueeze(2), saved=near[2])
    gb = ssd.selective_scan_backward(x, far[0], far[1], A, far[2].unsqueeze(2), far[3].unsqueeze(2), saved=got[2])
    assert all(torch.equal(a, b) for a, b in zip(ga, gb) if a is not None)
    for a, b in zip(ssd.causal_conv(x, w), ssd.causal_conv(far[0], w)):
        assert torch.equal(a, b)
    for a, b in zip(ssd.causal_conv_backward(x, x, w), ssd.causal_conv_backward(x, far[0], w)):
        assert a is None or torch.equal(a, b)
    del wide, far, v
    # pools: 2^31 elements and more
    D, N = 4096, 64
    slots = (1 << 31) // (D * N) + 3
    pool = torch.zeros(slots, D, N, dtype=torch.bfloat16, device="cuda")
    where = torch.tensor([slots - 1, 1], dtype=torch.int32, device="cuda")
    x = torch.randn(2, D, generator=g).bfloat16().cuda()
    B = torch.randn(2, 1, N, generator=g).bfloat16().cuda()
    A = -torch.ones(D, N, device="cuda")
    small = torch.zeros(2, D, N, dtype=torch.bfloat16, device="cuda")
    a = ssd.selective_scan_step(x, x, A, B, B, state=pool, slots=where)
    b = ssd.selective_scan_step(x, x, A, B, B, state=small)
    assert torch.equal(a, b) and torch.equal(pool[where.long()], small) and not pool[2:slots - 1:997].any()
    del pool
    codes, scales = ssd.state_cache(2 * slots, (D, N), group=32)
    where = torch.tensor([2 * slots - 1, 1], dtype=torch.int32, device="cuda")
    ssd.state_cache_write(small, codes, scales, where)
    back = ssd.state_cache_read(codes, scales, where, state_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert torch.equal(back.cpu(), ref.cache(small.cpu(), 32, "int8")[0].float().bfloat16())
    cpool = torch.zeros((1 << 31) // (D * 3) + 2, D, 3, dtype=torch.bfloat16, device="cuda")
    cw = torch.ones(D, 4, device="cuda")
    last = torch.tensor([cpool.shape[0] - 1, 0], dtype=torch.int32, device="cuda")
    ssd.causal_conv_step(x, cw, state=cpool, slots=last)
    assert torch.equal(cpool[last.long()][..., 2], x) and not cpool[1:-1:99991].any()


def test_threads_at_once():
    """Calls from several threads, each on its own stream, of sizes that are new to all of them."""
    import threading
    jobs = []
    for i in range(6):
        s, seq, S, _ = scan_inputs(2, 40 + 7 * (i // 2), 70, 16, 1, "bf16", "f32", "pad", True, True, True, True, seed=60 + i)
        args, h0 = call_args(s)
        w = torch.randn(70, 4, generator=gen(i)).cuda()
        jobs.append((args, h0, w, dict(seq_idx=seq.cuda(), nseq=S)))
    torch.cuda.synchronize()

    def work(args, h0, w, kw):
        out, fin, saved = ssd.selective_scan(*args, initial_state=h0, save_for_backward=True, **kw)
        g = ssd.selective_scan_backward(out, *args, saved=saved, initial_state=h0, **kw)
        c, cs = ssd.causal_conv(args[0], w, **kw)
        return [out, fin, *g, c, cs]

    got = [None] * len(jobs)

    def run(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(5):
                got[i] = work(*jobs[i])
        st.synchronize()
    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i, j in enumerate(jobs):
        for a, b in zip(got[i], work(*j)):
            assert (a is None and b is None) or torch.equal(a, b), i


def test_first_call_inside_a_capture():
    """Sizes not seen before, packed, in many time splits, captured at their first call and replayed."""
    L, D, N = 1537, 66, 32
    s, seq, S, g = scan_inputs(1, L, D, N, 1, "f16", "bf16", "pad", True, True, True, True, seed=71)
    args, h0 = call_args(s)
    kw = dict(seq_idx=seq.cuda(), nseq=S, initial_state=h0)
    dout = torch.randn(1, L, D, generator=g).half().cuda()
    w = torch.randn(D, 3, generator=g).cuda()
    torch.cuda.synchronize()

    def work():
        out, fin, saved = ssd.selective_scan(*args, save_for_backward=True, **kw)
        gr = ssd.selective_scan_backward(dout, *args, saved=saved, **kw)
        c, cs = ssd.causal_conv(args[0], w, seq_idx=kw["seq_idx"], nseq=S)
        cg = ssd.causal_conv_backward(dout, args[0], w, seq_idx=kw["seq_idx"], nseq=S)
        return [out, fin, *gr, c, cs, *cg]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for k in range(3):
        dout.copy_(torch.randn(1, L, D, generator=g).half())
        args[0].copy_(torch.randn(1, L, D, generator=g).half())
        graph.replay()
        torch.cuda.synchronize()
        got = [None if t is None else t.clone() for t in held]
        want = work()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert (a is None and b is None) or torch.equal(a, b), k


@pytest.mark.parametrize("L,D,N", [(60, 70, 16), (1700, 20, 8), (300, 40, 64)])
def test_padding_adds_nothing_to_gradients(L, D, N):
    """NaN and infinities in padded tokens, in every input and in dout: the gradients are those of clean padding, to the
    bit, and zero at the padding."""
    s, _, _, g = scan_inputs(2, L, D, N, 1, "bf16", "f32", None, False, True, True, True, seed=81)
    seq = torch.full((2, L), -1, dtype=torch.int32)
    seq[0, 5:L // 3], seq[0, L // 3:L // 3 + 9], seq[1, :2], seq[1, L - 20:] = 0, 1, 2, 3
    pad = seq < 0
    dout = torch.randn(2, L, D, generator=g).bfloat16()
    w, b = torch.randn(D, 4, generator=g).cuda(), torch.randn(D, generator=g).cuda()
    h0, c0 = torch.randn(4, D, N, generator=g).cuda(), torch.randn(4, D, 3, generator=g).bfloat16().cuda()
    dfin, dcfin = torch.randn(4, D, N, generator=g).cuda(), torch.randn(4, D, 3, generator=g).bfloat16().cuda()
    kw = dict(seq_idx=seq.cuda(), nseq=4)
    res = []
    for value in (0.0, float("nan"), float("inf"), float("-inf")):
        inp = {k: (None if t is None else t.clone()) for k, t in s.items()}
        do = dout.clone()
        do[pad] = value
        for k in ("x", "dt", "B", "C", "z"):
            inp[k][pad] = value
        args, _ = call_args(inp)
        saved = ssd.selective_scan(*args, initial_state=h0, save_for_backward=True, **kw)[2]
        gr = ssd.selective_scan_backward(do.cuda(), *args, saved=saved, initial_state=h0, dfinal_state=dfin, **kw)
        cg = ssd.causal_conv_backward(do.cuda(), args[0], w, b, initial_state=c0, dfinal_state=dcfin, **kw)
        torch.cuda.synchronize()
        res.append([*gr, *cg])
        for t in (gr.dx, gr.ddt, gr.dB, gr.dC, gr.dz, cg.dx):
            assert not t[pad.cuda()].any()
    for value, got in enumerate(res):
        for name, a, c in zip(gr._fields + cg._fields, got, res[0]):
            assert torch.isfinite(a.float()).all() and torch.equal(a, c), (value, name)


def test_steps_on_views_far_apart():
    """A token of every row of long tensors, both steps of a layer: views whose rows lie more than 2^24 elements apart."""
    B, D, N, row = 3, 64, 16, (1 << 24) + 128
    s, _, _, g = scan_inputs(B, 1, D, N, 1, "bf16", "f32", None, True, True, True, True, seed=91)
    (x, dt, A, Bm, C, Dp, bias, z), h0 = call_args(s)
    wide = torch.zeros(B, row, dtype=torch.bfloat16, device="cuda")
    near = [x[:, 0], dt[:, 0], Bm[:, 0], C[:, 0], z[:, 0]]
    far = [wide[:, 64 * i:64 * i + t[0].numel()].unflatten(1, t.shape[1:]) for i, t in enumerate(near)]
    for f, t in zip(far, near):
        f.copy_(t)
    pools, outs = [h0.clone(), h0.clone()], []
    for st, (x_, dt_, B_, C_, z_) in zip(pools, (near, far)):
        outs.append(ssd.selective_scan_step(x_, dt_, A, B_, C_, Dp, bias, z_, state=st))
    w, convs = torch.randn(D, 4, generator=g).cuda(), []
    for x_ in (near[0], far[0]):
        st = torch.zeros(B, D, 3, dtype=torch.bfloat16, device="cuda")
        convs += [ssd.causal_conv_step(x_, w, state=st), st]
    torch.cuda.synchronize()
    assert far[0].stride(0) == row and torch.equal(*outs) and torch.equal(*pools)
    assert torch.equal(convs[0], convs[2]) and torch.equal(convs[1], convs[3])
    check_scan((outs[1][:, None], pools[1]), s, B, True, ref.runs(B, 1), 1, N, "f32", "far step")


# Lanes take two batch rows once that leaves 1024 workgroups: ceil(D / (1024 / N)) * (B // 2) of them.
@pytest.mark.parametrize("N,D,G,B", [(16, 2048, 1, 65), (8, 4100, 2, 63), (32, 1028, 4, 65), (64, 520, 1, 64), (16, 2048, 2, 63),
                                     (8, 4100, 1, 64)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sdtype", ["f32", "f16", "bf16"])
def test_scan_step_of_large_batches(N, D, G, B, dtype, sdtype):
    """Batches at and below the edge (32 * 32, 33 * 31, 33 * 32, 33 * 32, 32 * 31, 33 * 32 workgroups), odd and even, on
    shuffled slots of a larger pool; rows without a slot, each with a live one beside it; other slots keep their bits."""
    say("scan step of a large batch", N, D, G, B, dtype, sdtype)
    gate = sdtype != "f16"
    s, _, _, g = scan_inputs(B, 1, D, N, G, dtype, sdtype, None, True, gate, gate, gate, seed=101)
    (x, dt, A, Bm, C, Dp, bias, z), h0 = call_args(s)
    nslots = B + 9
    pool = torch.randn(nslots, D, N, generator=g).to(DT[sdtype]).cuda()
    where = torch.randperm(nslots, generator=g)[:B]
    slots = where.to(torch.int32)
    none = {4: -1, 9: nslots, 20: -2 ** 31, 31: 2 ** 31 - 1, B - 1: -7}
    for b, v in none.items():
        slots[b] = v
    live = torch.tensor([b not in none for b in range(B)])
    pool[where[live].cuda()] = h0[live.cuda()]
    before = pool.clone()
    out = ssd.selective_scan_step(x[:, 0], dt[:, 0], A, Bm[:, 0], C[:, 0], Dp, bias, None if z is None else z[:, 0],
                                  state=pool, slots=slots.cuda(), dt_softplus=gate)
    torch.cuda.synchronize()
    out, pool, before = out.cpu(), pool.cpu(), before.cpu()
    assert not out[~live].any()
    rest = torch.ones(nslots, dtype=torch.bool)
    rest[where[live]] = False
    assert torch.equal(pool[rest], before[rest])
    part = {k: v[live] if v is not None and k in ("x", "dt", "B", "C", "z", "h0") else v for k, v in s.items()}
    n = int(live.sum())
    check_scan((out[live][:, None], pool[where[live]]), part, n, gate, ref.runs(n, 1), 1, N, sdtype, "step")


def time_splits(B, L, D, N, G, backward):
    """The number of time splits, from the workspace: a split holds its state and the sum of its steps, backward also its
    part of dA, dD and ddt_bias beside dB and dC of every channel block."""
    import ctypes
    lib = ssd.load_library()
    p = ssd.ScanParams(ctypes.sizeof(ssd.ScanParams), B, L, D, N, G, 0, 0, 1, 0, 0, 0, 0, 0, 0)
    if not backward:
        return max(1, round(lib.ssd_selective_scan_workspace_size(ctypes.byref(p)) / (B * D * (N + 1) * 4)))
    bc = 2 * B * G * ((D // G + 63) // 64) * L * N * 4
    n = lib.ssd_selective_scan_backward_workspace_size(ctypes.byref(p)) - bc
    one = B * D * (N + 2) * 4
    return 1 if n < 1.5 * one else round(n / (one + B * D * (N + 1) * 4))


@pytest.mark.parametrize("want,backward,B,D,N,G,dtype,sdtype", [
    (2, False, 1, 70, 64, 1, "f32", "f32"), (4, True, 1, 64, 8, 1, "f32", "f32"), (6, False, 2, 130, 8, 2, "f32", "f32"),
    (9, False, 1, 70, 16, 1, "f16", "f32"), (9, True, 2, 70, 16, 1, "bf16", "f32"), (13, False, 1, 40, 32, 1, "f32", "bf16"),
    (13, True, 2, 33, 64, 1, "bf16", "f32"), (16, True, 2, 20, 16, 1, "f32", "f32"), (17, True, 1, 20, 16, 1, "f32", "f32"),
    (16, False, 1, 20, 16, 1, "f32", "f32"), (17, False, 2, 20, 32, 1, "f32", "f32")])
def test_states_cross_time_splits(want, backward, B, D, N, G, dtype, sdtype):
    """Unpacked prompts in few splits (joined within the passes up to 16, by a launch of their own from 17), their states
    going in and the gradients of those coming out across all of them.  The length is the first whose number of splits
    is nearest to the one wanted.

    The steps' sum times |A| stays below 0.0125 L over a row, so what enters at one end is there at the other.  A split's
    decay, from a sum of steps with at most (16 + 34 tiles) roundings, adds 0.0125 L * 50 u < L u to the 8 L u of the
    bound's exponentials, which count 8 roundings a token where two products, a sum and an exponential round 5 times."""
    L = min(range(33, 530), key=lambda n: (abs(time_splits(B, n, D, N, G, backward) - want), n))
    took = [time_splits(B, L, D, N, G, b) for b in (False, True)]
    say("states cross splits", want, backward, B, L, D, N, G, dtype, sdtype, "splits", took)
    assert took[backward] >= 2
    s, _, _, g = scan_inputs(B, L, D, N, G, dtype, sdtype, None, True, True, True, True, seed=111)
    s["A"] = -0.02 * torch.rand(D, N, generator=g)
    assert float(0.02 * ref.steps(s["dt"], s["bias"], True)[1].sum(1).max()) <= 0.0125 * L
    args, h0 = call_args(s)
    kw = dict(initial_state=h0, state_dtype=DT[sdtype])
    out, fin, saved = ssd.selective_scan(*args, save_for_backward=True, **kw)
    dout, dfin = torch.randn(B, L, D, generator=g).to(s["x"].dtype), torch.randn(B, D, N, generator=g).to(DT[sdtype])
    grads = ssd.selective_scan_backward(dout.cuda(), *args, saved=saved, dfinal_state=dfin.cuda(), **kw)
    torch.cuda.synchronize()
    rr = ref.runs(B, L)
    check_scan((out, fin), s, B, True, rr, L, N, sdtype, "splits")
    check_grads(grads, dout, dfin, s, B, True, rr, (B, L, D, N, G, dtype, sdtype))


def test_arguments_that_change_in_place():
    """A flag and a count held as tensors: a call reads their values of its own time."""
    s, seq, S, _ = scan_inputs(1, 20, 64, 16, 1, "f32", "f32", "pad", False, True, True, True, seed=121)
    args, _ = call_args(s)
    flag, n = torch.tensor(True), torch.tensor(S)
    plain = ssd.selective_scan(*args)
    for value, more in ((True, 0), (False, 2)):
        flag.fill_(value)
        n.fill_(S + more)
        a, b = (ssd.selective_scan(*args, dt_softplus=f, seq_idx=seq.cuda(), nseq=k) for f, k in ((flag, n), (value, S + more)))
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and len(a[1]) == S + more
    assert torch.isfinite(plain[0]).all()


def test_autograd_sees_what_is_written_in_place():
    """A state that torch's autograd holds for a backward pass and that a step then moves on: the backward refuses, as
    after a write by torch, and so for every tensor that a call writes into."""
    B, D, N = 2, 64, 16
    s, _, _, _ = scan_inputs(B, 1, D, N, 1, "f32", "f32", None, True, True, True, True, seed=131)
    (x, dt, A, Bm, C, Dp, bias, z), h0 = call_args(s)
    token = (x[:, 0], dt[:, 0], A, Bm[:, 0], C[:, 0], Dp, bias, z[:, 0])
    w = torch.ones(D, 4, device="cuda")
    new = lambda *shape: torch.zeros(*shape, device="cuda")  # noqa: E731
    codes, scales = ssd.state_cache(B, (D, N), group=16)
    state, conv, out, tok, fin, cfin, back = h0.clone(), new(B, D, 3), new(B, 1, D), new(B, D), new(B, D, N), new(B, D, 3), new(B, D, N)

    def calls():
        ssd.selective_scan_step(*token, state=state, out=tok)
        ssd.causal_conv_step(x[:, 0], w, state=conv)
        ssd.selective_scan(x, dt, A, Bm, C, Dp, bias, z, out=out, final_state=fin)
        ssd.causal_conv(x, w, final_state=cfin)
        ssd.state_cache_write(fin, codes, scales)
        ssd.state_cache_read(codes, scales, out=back)
    written = [state, conv, out, tok, fin, cfin, codes, scales, back]
    read = [x, dt, A, Bm, C, Dp, bias, z, w]
    before = [t._version for t in written], [t._version for t in read]
    calls()
    assert all(t._version > v for t, v in zip(written, before[0])) and [t._version for t in read] == before[1]
    p = torch.ones(B, D, N, device="cuda", requires_grad=True)
    loss = (p * state).sum()
    ssd.selective_scan_step(*token, state=state)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    with torch.inference_mode():
        state, out, tok, fin = state.clone(), new(B, 1, D), new(B, D), new(B, D, N)
        calls()
    torch.cuda.synchronize()


@pytest.mark.parametrize("L,pack", [(21, None), (21, "pad"), (131, None), (700, "full")])
def test_infinite_decays(L, pack):
    """A of -inf (and one whose product with log2(e) overflows) forgets the state at every step: outputs, states and gradients
    are those of the limit, which the 64-bit loops reach with A = -1e30, also in rows that end inside a tile."""
    B, D, N = 2, 66, 16
    s, seq, S, g = scan_inputs(B, L, D, N, 1, "f32", "f32", pack, True, True, True, True, seed=141)
    far = dict(s, A=s["A"].clone())
    for t, v in ((s["A"], -1e30), (far["A"], float("-inf"))):
        t[3, 5], t[65], t[7, 2] = v, v, -3.4e38
    args, h0 = call_args(far)
    kw = dict(seq_idx=cuda(seq), nseq=S if pack else None, initial_state=h0)
    out, fin, saved = ssd.selective_scan(*args, save_for_backward=True, **kw)
    dout, dfin = torch.randn(B, L, D, generator=g), torch.randn(S, D, N, generator=g)
    grads = ssd.selective_scan_backward(dout.cuda(), *args, saved=saved, dfinal_state=dfin.cuda(), **kw)
    torch.cuda.synchronize()
    rr = ref.runs(B, L, seq)
    check_scan((out, fin), s, S, True, rr, min(L, 400), N, "f32", "infinite decays")
    check_grads(grads, used(dout, seq, S), dfin, s, S, True, rr, (B, L, D, N, 1, "f32", "f32"))
