"""What stands around a mixer in a layer, and a second mixer: the root-mean-square norm with the residual's addition (its
output also in 8 bits), the matrix product with bias, activation and residual, and the gated linear recurrence.

A binding over the last part of include/mamba_ssd.h, in the manner of selective.py, whose conventions hold here too:
rows that are views, packed sequences (``seq_idx``, ``nseq``), pools of states (``slots``), the current stream of the
tensors' device, no autograd graph, raised version counters.  The names are re-exported by the package:

    y, s = rms_norm(x, norm_w, residual)                                 # s = x + residual
    xz = linear(y, in_w)
    xc, conv_state = causal_conv(xz[..., :D], conv_w, conv_b)            # (or a selective scan behind it)
    h, state = gated_recurrence(xc, xz[..., D:2 * D], A, xz[..., 2 * D:], gate_b, in_b)
    s = linear(h, out_w, residual=s)

    codes, scales, s = rms_norm(x, norm_w, residual, format="e4m3")      # in 8 bits, a scale a row
    xz = linear(codes, in_codes, x_scale=scales, weight_scale=in_scales, out_dtype=x.dtype)

    out_t = gated_recurrence_step(x_t, gate_t, A, in_t, gate_b, in_b, state=state)      # one token, in place

    h, _, saved = gated_recurrence(..., save_for_backward=True)          # training
    g = gated_recurrence_backward(dout, ..., saved=saved)                # g.dx, g.dgate, g.dA, ...
    out, pre = linear(x, w, b, activation="silu", save_pre=True)
    g = linear_backward(dout, x, w, pre=pre, activation="silu", with_bias=True)         # g.dx, g.dweight, g.dbias
    g = rms_norm_backward(dout, s, norm_w, dresidual=ds)                 # g.dx, g.dresidual, g.dweight

Training keeps for the recurrence a state in fp32 every 64 tokens, for a product with an activation ``pre``, for the norm
the sum that it returns.
"""
import collections
import ctypes

from . import selective as _s

__all__ = ["rms_norm", "rms_norm_backward", "linear", "linear_backward", "gated_recurrence", "gated_recurrence_backward",
           "gated_recurrence_step", "NormGrads", "LinearGrads", "RecurrenceGrads", "NormParams", "LinearParams",
           "RecurrenceParams", "IN_INT8", "IN_E4M3"]

IN_INT8, IN_E4M3 = 3, 4
_FORMATS = {None: -1, "int8": _s.CACHE_INT8, "e4m3": _s.CACHE_E4M3}
_ACTS = {None: 0, "silu": 1, "gelu": 2}

NormGrads = collections.namedtuple("NormGrads", "dx dresidual dweight")
LinearGrads = collections.namedtuple("LinearGrads", "dx dweight dbias")
RecurrenceGrads = collections.namedtuple("RecurrenceGrads", "dx dgate dA din_gate dgate_bias din_bias dinitial_state")


class NormParams(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_size_t), ("rows", ctypes.c_int64), ("width", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("sum_dtype", ctypes.c_int), ("format", ctypes.c_int), ("eps", ctypes.c_float),
                ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64)]


class LinearParams(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_size_t), ("rows", ctypes.c_int), ("width", ctypes.c_int), ("outs", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("act", ctypes.c_int), ("x_stride", ctypes.c_int64),
                ("residual_stride", ctypes.c_int64)]


class RecurrenceParams(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_size_t), ("batch", ctypes.c_int), ("seqlen", ctypes.c_int),
                ("channels", ctypes.c_int), ("in_dtype", ctypes.c_int), ("state_dtype", ctypes.c_int),
                ("normalize", ctypes.c_int), ("nseq", ctypes.c_int), ("x_stride", ctypes.c_int64),
                ("gate_stride", ctypes.c_int64), ("in_stride", ctypes.c_int64)]


# (pointers after the parameter block, and whether workspace, workspace_bytes follow)
_SIGNATURES = {"ssd_rms_norm": (NormParams, 6, False), "ssd_rms_norm_backward": (NormParams, 7, True),
               "ssd_linear": (LinearParams, 8, True), "ssd_linear_backward": (LinearParams, 7, True),
               "ssd_gated_recurrence": (RecurrenceParams, 11, True),
               "ssd_gated_recurrence_backward": (RecurrenceParams, 18, True),
               "ssd_gated_recurrence_step": (RecurrenceParams, 9, False)}
_SIZES = {"ssd_rms_norm_backward_workspace_size": NormParams, "ssd_linear_workspace_size": LinearParams,
          "ssd_linear_backward_workspace_size": LinearParams, "ssd_gated_recurrence_workspace_size": RecurrenceParams,
          "ssd_gated_recurrence_saved_size": RecurrenceParams,
          "ssd_gated_recurrence_backward_workspace_size": RecurrenceParams}
EXPORTED_SYMBOLS = sorted(_SIGNATURES) + sorted(_SIZES)


def declare(lib):
    """Argument types of this module's entry points (called once, when the library is loaded)."""
    _s.declare(lib, _SIGNATURES, _SIZES)


# ---- helpers -------------------------------------------------------------------------------------
def _lead(x, what):
    """Leading dimensions of a tensor of rows, and how many rows these are."""
    if x.dim() < 2:
        raise ValueError("%s must have at least 2 dimensions (got %d)" % (what, x.dim()))
    n = 1
    for d in x.shape[:-1]:
        n *= d
    return tuple(x.shape[:-1]), n


def _counts(**sizes):
    """Sizes that a parameter block holds in 32 bits (ctypes would cut them)."""
    for name, n in sizes.items():
        if n >= 2**31:
            raise ValueError("%s must be below 2^31 (got %d)" % (name, n))


def _workspace(plan, given, i=0):
    return _s._new(plan.spaces[i])[0] if given is None else _s._space(given, plan.dev)


# ---- residual norm --------------------------------------------------------------------------------
def _norm_params(x, weight, residual, sum_dtype, eps, fmt):
    dev = _s._on_gpu(x, "rms_norm")
    lead, rows = _lead(x, "x")
    D = x.shape[-1]
    import torch
    _counts(width=D)
    _s._same(dev, torch.float32, weight=(weight, (D,)))
    xs = _s._rows("x", x, dev, x.dtype, x.shape, len(lead))
    rs = 0 if residual is None else _s._rows("residual", residual, dev, sum_dtype, x.shape, len(lead))
    return NormParams(ctypes.sizeof(NormParams), rows, D, 0, _s._state_code(sum_dtype), _FORMATS[fmt], eps, xs, rs), dev, lead


def _norm_plan(x, weight, residual, eps, fmt, out, residual_out):
    import torch
    code = _s._code(x, "x")
    sum_dtype = x.dtype if residual is None else residual.dtype
    if sum_dtype not in (x.dtype, torch.float32):
        raise ValueError("residual must be %s or float32 (got %s)" % (x.dtype, sum_dtype))
    if fmt not in _FORMATS:
        raise ValueError("format must be None, 'int8' or 'e4m3'")
    prm, dev, lead = _norm_params(x, weight, residual, sum_dtype, eps, fmt)
    prm.in_dtype = code
    dtype = {None: x.dtype, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[fmt]
    _s._same(dev, dtype, out=(out, x.shape))
    if residual_out is not None and residual is None:
        raise ValueError("residual_out goes with residual")
    _s._same(dev, sum_dtype, residual_out=(residual_out, x.shape))
    return _s._Plan("ssd_rms_norm", prm, dev, _s._layout(x.shape, dtype, dev), state=_s._layout(x.shape, sum_dtype, dev),
                    new=_s._layout(lead, torch.float32, dev))


def rms_norm(x, weight, residual=None, *, eps=1e-5, format=None, out=None, residual_out=None):
    """ssd_rms_norm: the root-mean-square norm of the rows of x + residual, x [..., D] (float32, float16 or bfloat16,
    D <= 16384), weight [D] float32, residual [..., D] of x's type or float32.  Returns out [..., D]; with a residual
    (out, sum), the sum in the residual's type; with ``format`` "int8" or "e4m3" codes [..., D] (torch.int8 or
    torch.float8_e4m3fn) and scales [...] float32 in the place of out.  ``residual_out`` may be the (contiguous)
    residual itself."""
    meta, (px, pw, pr, _, _) = _s._meta(x, weight, residual, out, residual_out)
    key = ("norm", meta, eps, format)
    plan = _s._PLANS.get(key) or _s._older(key)
    if plan is None:
        plan = _s._keep(key, _norm_plan(x, weight, residual, eps, format, out, residual_out))
    if out is None and residual is not None and residual_out is None:
        out, residual_out = _s._new(plan.out, plan.state)
    elif out is None:
        out, = _s._new(plan.out)
    elif residual is not None and residual_out is None:
        residual_out, = _s._new(plan.state)
    scales = None if format is None else _s._new(plan.new)[0]
    plan.call(px, pw, pr, out, scales, residual_out)
    got = (out,) if format is None else (out, scales)
    if residual is not None:
        got += (residual_out,)
    return got if len(got) > 1 else out


def _norm_backward_plan(dout, s, weight, eps, dresidual):
    import torch
    code = _s._code(dout, "dout")
    if s.dtype not in (dout.dtype, torch.float32):
        raise ValueError("s must be %s or float32 (got %s)" % (dout.dtype, s.dtype))
    prm, dev, _ = _norm_params(s, weight, None, s.dtype, eps, None)
    prm.in_dtype = code
    _s._same(dev, dout.dtype, dout=(dout, s.shape))
    _s._same(dev, s.dtype, dresidual=(dresidual, s.shape))
    lay = lambda t, like=s: _s._layout(like.shape, t, dev)  # noqa: E731
    return _s._Plan("ssd_rms_norm_backward", prm, dev, lay(dout.dtype), None if s.dtype == dout.dtype else lay(s.dtype),
                    lay(torch.float32, weight), ("ssd_rms_norm_backward_workspace_size",))


def rms_norm_backward(dout, s, weight, *, eps=1e-5, dresidual=None, workspace=None):
    """ssd_rms_norm_backward: NormGrads(dx, dresidual, dweight) of rms_norm at ``s``, the sum that it returned (x where
    there was no residual), from the gradient of its output and, if given, that of the sum (``dresidual``).  dx has
    dout's type and dresidual that of s: one tensor where these are the same."""
    meta, (pg, ps, pw, pd) = _s._meta(dout, s, weight, dresidual)
    key = ("norm backward", meta, eps)
    plan = _s._PLANS.get(key) or _s._older(key)
    if plan is None:
        plan = _s._keep(key, _norm_backward_plan(dout, s, weight, eps, dresidual))
    dx, dw, space, *dr = _s._new(plan.out, plan.state, plan.spaces[0], *([] if plan.parts is None else [plan.parts]))
    workspace = space if workspace is None else _s._space(workspace, plan.dev)
    plan.call(pg, ps, pw, pd, dx, dr[0] if dr else None, dw, workspace, workspace.numel())
    return NormGrads(dx, dr[0] if dr else dx, dw)


# ---- matrix product -------------------------------------------------------------------------------
def _linear_params(x, weight, act, out_dtype, what):
    import torch
    dev = _s._on_gpu(x, what)
    codes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int8: IN_INT8, torch.float8_e4m3fn: IN_E4M3}
    if x.dtype not in codes:
        raise ValueError("x must be float32, float16, bfloat16, int8 or float8_e4m3fn (got %s)" % x.dtype)
    if act not in _ACTS:
        raise ValueError("activation must be None, 'silu' or 'gelu'")
    lead, rows = _lead(x, "x")
    if weight.dim() != 2:
        raise ValueError("weight must be [outs, width]")
    K, N = x.shape[-1], weight.shape[0]
    _counts(rows=rows, width=K, outs=N)
    _s._same(dev, x.dtype, weight=(weight, (N, K)))
    xs = _s._rows("x", x, dev, x.dtype, x.shape, len(lead))
    return LinearParams(ctypes.sizeof(LinearParams), rows, K, N, codes[x.dtype], _s._state_code(out_dtype), _ACTS[act], xs,
                        0), dev, lead


def _linear_plan(x, weight, bias, residual, act, x_scale, weight_scale, out_dtype, out, off):
    import torch
    if out_dtype is None:
        given = [t for t in (out, residual) if t is not None]
        if x.dtype.itemsize == 1 and not given:
            raise ValueError("operands in 8 bits need out_dtype")
        out_dtype = given[0].dtype if given else x.dtype
    prm, dev, lead = _linear_params(x, weight, act, out_dtype, "linear")
    N = prm.outs
    if off and not prm.x_stride:  # rows of a view, as the library sees it: they may start anywhere
        prm.x_stride = prm.width
    _s._same(dev, torch.float32, bias=(bias, (N,)), x_scale=(x_scale, lead), weight_scale=(weight_scale, (N,)))
    if residual is not None:
        prm.residual_stride = _s._rows("residual", residual, dev, out_dtype, lead + (N,), len(lead))
    _s._same(dev, out_dtype, out=(out, lead + (N,)))
    return _s._Plan("ssd_linear", prm, dev, _s._layout(lead + (N,), out_dtype, dev), spaces=("ssd_linear_workspace_size",))


def linear(x, weight, bias=None, residual=None, *, activation=None, x_scale=None, weight_scale=None, out_dtype=None,
           save_pre=False, out=None, workspace=None):
    """ssd_linear: act(x weight^T + bias) + residual, x [..., K], weight [N, K], bias [N] float32, residual [..., N];
    ``activation`` None, "silu" or "gelu".  x and weight are float32, float16 or bfloat16, or 8-bit codes (torch.int8,
    torch.float8_e4m3fn) with ``x_scale`` [...] and ``weight_scale`` [N] float32 (None: 1); e4m3 has sums of full fp32
    precision where ``out_dtype`` is float32.  Returns out [..., N] in
    ``out_dtype`` (default: out's, the residual's, or x's), and with ``save_pre`` (out, pre) for linear_backward.  ``out`` may
    be the (contiguous) residual itself."""
    meta, (px, pw, pb, pr, psx, psw, _) = _s._meta(x, weight, bias, residual, x_scale, weight_scale, out)
    off = px & 15 != 0  # contiguous rows of a view: one row of a batch, or ones behind an odd offset
    key = ("linear", meta, activation, out_dtype, off)
    plan = _s._PLANS.get(key) or _s._older(key)
    if plan is None:
        plan = _s._keep(key, _linear_plan(x, weight, bias, residual, activation, x_scale, weight_scale, out_dtype, out, off))
    if out is None and workspace is None:
        out, workspace = _s._new(plan.out, plan.spaces[0])
    else:
        out = _s._new(plan.out)[0] if out is None else out
        workspace = _workspace(plan, workspace)
    pre = _s._new(plan.out)[0] if save_pre else None
    plan.call(px, pw, pb, pr, psx, psw, pre, out, workspace, workspace.numel())
    return (out, pre) if save_pre else out


def _linear_backward_plan(dout, x, weight, pre, act):
    import torch
    if x.dtype.itemsize == 1:
        raise ValueError("linear_backward takes float32, float16 and bfloat16 (got %s)" % x.dtype)
    prm, dev, lead = _linear_params(x, weight, act, x.dtype, "linear_backward")
    _s._same(dev, x.dtype, dout=(dout, lead + (prm.outs,)), pre=(pre, lead + (prm.outs,)))
    if (pre is None) != (act is None):
        raise ValueError("pre goes with an activation")
    return _s._Plan("ssd_linear_backward", prm, dev, _s._layout(x.shape, x.dtype, dev),
                    _s._layout(weight.shape, x.dtype, dev), _s._layout((prm.outs,), torch.float32, dev),
                    ("ssd_linear_backward_workspace_size",))


def linear_backward(dout, x, weight, *, pre=None, activation=None, with_bias=False, with_dx=True, with_dweight=True,
                    workspace=None):
    """ssd_linear_backward: LinearGrads(dx, dweight, dbias) of linear from the gradient of its output (which is the
    residual's too), its inputs and, with an activation, the ``pre`` that it returned.  Those not wanted are None."""
    meta, (pg, px, pw, pp) = _s._meta(dout, x, weight, pre)
    key = ("linear backward", meta, activation)
    plan = _s._PLANS.get(key) or _s._older(key)
    if plan is None:
        plan = _s._keep(key, _linear_backward_plan(dout, x, weight, pre, activation))
    dx = _s._new(plan.out)[0] if with_dx else None
    dw = _s._new(plan.parts)[0] if with_dweight else None
    db = _s._new(plan.state)[0] if with_bias else None
    workspace = _workspace(plan, workspace)
    plan.call(pg, px, pw, pp, dx, dw, db, workspace, workspace.numel())
    return LinearGrads(dx, dw, db)


# ---- gated recurrence -------------------------------------------------------------------------------
def _recurrence_params(x, gate, A, in_gate, gate_bias, in_bias, normalize, state_code, nseq, lead):
    import torch
    dev = _s._on_gpu(x, "gated_recurrence")
    if x.dim() != len(lead) + 1:
        raise ValueError("x must have %d dimensions (got %d)" % (len(lead) + 1, x.dim()))
    code, ch = _s._code(x, "x"), x.shape[-1]
    _counts(batch=lead[0], seqlen=lead[-1] if len(lead) > 1 else 1, channels=ch, nseq=nseq)
    _s._same(dev, torch.float32, A=(A, (ch,)), gate_bias=(gate_bias, (ch,)), in_bias=(in_bias, (ch,)))
    if in_bias is not None and in_gate is None:
        raise ValueError("in_bias goes with in_gate")
    rows = lambda name, t: 0 if t is None else _s._rows(name, t, dev, x.dtype, lead + (ch,), len(lead))  # noqa: E731
    return RecurrenceParams(ctypes.sizeof(RecurrenceParams), lead[0], lead[1] if len(lead) > 1 else 1, ch, code, state_code,
                            1 if normalize else 0, nseq, rows("x", x), rows("gate", gate), rows("in_gate", in_gate)), dev


def _recurrence_plan(name, spaces, x, gate, A, in_gate, gate_bias, in_bias, normalize, seq_idx, nseq, state_dtype, states,
                     like_x):
    import torch
    lead = tuple(x.shape[:2])
    S = _s._seq(seq_idx, nseq, lead, x.device)
    if state_dtype is None:
        given = [t for t in states.values() if t is not None]
        state_dtype = given[0].dtype if given else torch.float32
    prm, dev = _recurrence_params(x, gate, A, in_gate, gate_bias, in_bias, normalize, _s._state_code(state_dtype), S, lead)
    _s._same(dev, torch.int32, seq_idx=(seq_idx, lead))
    state = (S, prm.channels)
    for n, t in states.items():
        _s._same(dev, state_dtype, **{n: (t, state)})
    for n, t in like_x.items():
        _s._same(dev, x.dtype, **{n: (t, x.shape)})
    lay = lambda t: None if t is None else _s._layout(t.shape, t.dtype, dev)  # noqa: E731
    return _s._Plan(name, prm, dev, lay(x), state=_s._layout(state, state_dtype, dev), spaces=spaces,
                    new=[lay(t) for t in (x, gate, A, in_gate, gate_bias, in_bias)])


def gated_recurrence(x, gate, A, in_gate=None, gate_bias=None, in_bias=None, *, normalize=True, seq_idx=None, nseq=None,
                     initial_state=None, state_dtype=None, save_for_backward=False, with_final_state=True, final_state=None,
                     out=None, workspace=None):
    """ssd_gated_recurrence over a prompt: h = a h + beta i x with a = exp(A sigmoid(gate + gate_bias)),
    i = sigmoid(in_gate + in_bias) (1 without in_gate) and beta = sqrt(1 - a^2) (1 without ``normalize``); x, gate, in_gate
    [B, L, D], A (<= 0) and the biases [D] float32.  Returns (out [B, L, D], final_state [B or nseq, D]), and with
    ``save_for_backward`` a third tensor for gated_recurrence_backward.  ``state_dtype`` defaults to initial_state's,
    else float32."""
    meta, (px, pg, pA, pi, pgb, pib, ps, ph, _, _) = _s._meta(x, gate, A, in_gate, gate_bias, in_bias, seq_idx, initial_state,
                                                              final_state, out)
    key = ("recurrence", meta, normalize, nseq, state_dtype)
    plan = _s._PLANS.get(key) or _s._older(key)
    if plan is None:
        plan = _s._keep(key, _recurrence_plan("ssd_gated_recurrence", ("ssd_gated_recurrence_workspace_size",
                                                                       "ssd_gated_recurrence_saved_size"),
                                              x, gate, A, in_gate, gate_bias, in_bias, normalize, seq_idx, nseq, state_dtype,
                                              dict(initial_state=initial_state, final_state=final_state), dict(out=out)))
    if out is None:
        out, = _s._new(plan.out)
    if final_state is None and with_final_state:
        final_state = _s._states(seq_idx is not None, plan.state)
    workspace = _workspace(plan, workspace)
    saved = _s._new(plan.spaces[1])[0] if save_for_backward else None
    plan.call(px, pg, pA, pi, pgb, pib, ps, ph, out, final_state, saved, workspace, workspace.numel())
    return (out, final_state, saved) if save_for_backward else (out, final_state)


def gated_recurrence_backward(dout, x, gate, A, in_gate=None, gate_bias=None, in_bias=None, *, saved, normalize=True,
                              seq_idx=None, nseq=None, initial_state=None, dfinal_state=None, state_dtype=None,
                              workspace=None):
    """ssd_gated_recurrence_backward: RecurrenceGrads of gated_recurrence from dout [B, L, D], dfinal_state (None: zeros),
    the forward's inputs and the ``saved`` tensor it returned.  din_gate, dgate_bias, din_bias and dinitial_state are
    None where the input is."""
    import torch
    meta, (pd, px, pg, pA, pi, pgb, pib, ps, ph, pf, psv) = _s._meta(dout, x, gate, A, in_gate, gate_bias, in_bias, seq_idx,
                                                                     initial_state, dfinal_state, saved)
    key = ("recurrence backward", meta, normalize, nseq, state_dtype)
    plan = _s._PLANS.get(key) or _s._older(key)
    if plan is None:
        plan = _recurrence_plan("ssd_gated_recurrence_backward", ("ssd_gated_recurrence_backward_workspace_size",
                                                                  "ssd_gated_recurrence_saved_size"),
                                x, gate, A, in_gate, gate_bias, in_bias, normalize, seq_idx, nseq, state_dtype,
                                dict(initial_state=initial_state, dfinal_state=dfinal_state), dict(dout=dout))
        _s._same(plan.dev, torch.uint8, saved=(saved, (plan.sizes[1],)))
        _s._keep(key, plan)
    made = iter(_s._new(*[n for n in plan.new if n is not None]))
    g = RecurrenceGrads(*[None if n is None else next(made) for n in plan.new],
                        None if initial_state is None else _s._states(seq_idx is not None, plan.state))
    workspace = _workspace(plan, workspace)
    plan.call(pd, pf, px, pg, pA, pi, pgb, pib, ps, ph, psv, *g, workspace, workspace.numel())
    return g


def _recurrence_step_plan(x, gate, A, in_gate, gate_bias, in_bias, state, slots, normalize, out):
    import torch
    lead = tuple(x.shape[:1])
    if state.dim() != 2:
        raise ValueError("state must be [nslots, channels]")
    prm, dev = _recurrence_params(x, gate, A, in_gate, gate_bias, in_bias, normalize, _s._state_code(state.dtype),
                                  state.shape[0], lead)
    _s._same(dev, state.dtype, state=(state, (state.shape[0], prm.channels)))
    _s._same(dev, torch.int32, slots=(slots, lead))
    _s._same(dev, x.dtype, out=(out, x.shape))
    return _s._Plan("ssd_gated_recurrence_step", prm, dev, _s._layout(x.shape, x.dtype, dev))


def gated_recurrence_step(x, gate, A, in_gate=None, gate_bias=None, in_bias=None, *, state, slots=None, normalize=True,
                          out=None):
    """ssd_gated_recurrence_step: one token per row; x, gate, in_gate [B, D].  ``state`` [nslots, D] is updated in place;
    row b uses state ``slots[b]`` (int32; None: state b).  A row whose slot is not in [0, nslots) touches no state
    and returns zeros.  Returns out [B, D]."""
    meta, (px, pg, pA, pi, pgb, pib, _, psl, _) = _s._meta(x, gate, A, in_gate, gate_bias, in_bias, state, slots, out)
    key = ("recurrence step", meta, normalize)
    plan = _s._PLANS.get(key) or _s._older(key)
    if plan is None:
        plan = _s._keep(key, _recurrence_step_plan(x, gate, A, in_gate, gate_bias, in_bias, state, slots, normalize, out))
    if out is None:
        out, = _s._new(plan.out)
    plan.call(px, pg, pA, pi, pgb, pib, state, psl, out)
    return out
