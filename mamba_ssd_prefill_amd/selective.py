"""The selective state space scan, its short causal convolution and the 8-bit state cache.

A binding over the second half of include/mamba_ssd.h, in the manner of the package's other entry
points: it checks arguments, allocates outputs and workspaces, and passes pointers and the current
stream of the tensors' device.  The calls themselves go through a small compiled module (_meta, built
beside the library against torch's headers).  The names are re-exported by the package:

    xc, conv_state = causal_conv(x, conv_w, conv_b)                      # prompt
    out, state = selective_scan(xc, dt, A, B, C, D, dt_bias, z)
    xt = causal_conv_step(x_t, conv_w, conv_b, state=conv_state)         # then token by token, in place
    out_t = selective_scan_step(xt, dt_t, A, B_t, C_t, D, dt_bias, z_t, state=state)

    out, _, saved = selective_scan(..., save_for_backward=True)          # training
    g = selective_scan_backward(dout, ..., saved=saved)                  # g.dx, g.ddt, g.dA, ...

    codes, scales = state_cache(nslots, (H, P, N))                       # states in 8 bits
    state_cache_write(state, codes, scales, slots)
    state = state_cache_read(codes, scales, slots)

Inputs with one row per token (x, dt, z, B, C) may be views whose rows lie a constant distance apart,
such as the halves of a joint projection; everything else is contiguous.  Outputs that are handed in
(``out``, ``final_state``) overlap no input.  Sequences packed into a
batch row are told apart by ``seq_idx`` (int32 [B, L], numbers in [0, nseq), each for one run of tokens;
-1: padding, which gets and adds zero gradients), and states then have one entry per number instead
of one per batch row.  ``slots`` name each state that a call writes once.

These calls are outside torch's autograd: what they return carries no graph, whether or not the inputs require
gradients; gradients come from the _backward calls (wrap a pair in a torch.autograd.Function to train through
them).  Tensors that a call writes in place (states, ``out``, ``final_state``, codes and scales) raise their version
counters as torch's own writes do.

Training keeps ``saved``: a state in fp32 every 8 tokens, 4 * B * ceil(L / 8) * D * N bytes.  That is N / 4
times a 16-bit x: 4 times at N = 16, 671 MB for one layer at 2 x 8192 x 5120.
"""
import collections
import ctypes
import numbers
import struct

from . import SSDError, _dtype_code, load_library

__all__ = ["causal_conv", "causal_conv_backward", "causal_conv_step", "selective_scan", "selective_scan_backward",
           "selective_scan_step", "state_cache", "state_cache_write", "state_cache_read", "ConvGrads", "ScanGrads",
           "ConvParams", "ScanParams", "CacheParams", "CACHE_INT8", "CACHE_E4M3"]

CACHE_INT8, CACHE_E4M3 = 0, 1

ConvGrads = collections.namedtuple("ConvGrads", "dx dweight dbias dinitial_state")
ScanGrads = collections.namedtuple("ScanGrads", "dx ddt dA dB dC dD ddt_bias dz dinitial_state")


class ConvParams(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_size_t), ("batch", ctypes.c_int), ("seqlen", ctypes.c_int),
                ("channels", ctypes.c_int), ("width", ctypes.c_int), ("in_dtype", ctypes.c_int), ("silu", ctypes.c_int),
                ("nseq", ctypes.c_int), ("split_a", ctypes.c_int), ("split_b", ctypes.c_int),
                ("x_stride", ctypes.c_int64)]


class ScanParams(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_size_t), ("batch", ctypes.c_int), ("seqlen", ctypes.c_int),
                ("channels", ctypes.c_int), ("dstate", ctypes.c_int), ("ngroups", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("state_dtype", ctypes.c_int), ("dt_softplus", ctypes.c_int),
                ("nseq", ctypes.c_int), ("x_stride", ctypes.c_int64), ("dt_stride", ctypes.c_int64),
                ("z_stride", ctypes.c_int64), ("B_stride", ctypes.c_int64), ("C_stride", ctypes.c_int64)]


class CacheParams(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_size_t), ("batch", ctypes.c_int), ("nslots", ctypes.c_int),
                ("elems", ctypes.c_int64), ("group", ctypes.c_int), ("format", ctypes.c_int),
                ("state_dtype", ctypes.c_int)]


# (pointers after the parameter block; "w" marks the place of workspace, workspace_bytes)
_SIGNATURES = {"ssd_causal_conv": (ConvParams, 9, False), "ssd_causal_conv_backward": (ConvParams, 13, True),
               "ssd_causal_conv_step": (ConvParams, 8, False), "ssd_selective_scan": (ScanParams, 13, True),
               "ssd_selective_scan_backward": (ScanParams, 22, True), "ssd_selective_scan_step": (ScanParams, 11, False),
               "ssd_state_cache_write": (CacheParams, 4, False), "ssd_state_cache_read": (CacheParams, 4, False)}
_SIZES = {"ssd_causal_conv_backward_workspace_size": ConvParams, "ssd_selective_scan_workspace_size": ScanParams,
          "ssd_selective_scan_saved_size": ScanParams, "ssd_selective_scan_backward_workspace_size": ScanParams}
EXPORTED_SYMBOLS = sorted(_SIGNATURES) + sorted(_SIZES)


def declare(lib):
    """Argument types of this module's entry points (called once, when the library is loaded)."""
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    for name, (params, n, ws) in _SIGNATURES.items():
        f = getattr(lib, name)
        f.argtypes = [ctypes.POINTER(params)] + [vp] * n + ([vp, sz] if ws else []) + [vp]
        f.restype = ctypes.c_int
    for name, params in _SIZES.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = [ctypes.POINTER(params)], sz


# ---- helpers -------------------------------------------------------------------------------------
# A call's checks depend on its arguments' shapes, strides, types and devices alone, so their outcome -- a plan: the
# parameter block, the output layouts, the workspace size -- is kept under those and found again in a microsecond.
# Nothing is kept about a tensor's identity, address or contents.  Plans come in two generations: when the newer one is
# full the older one goes, and a plan found in the older one moves on, so that those in use stay.
_PLANS, _BEFORE = {}, {}
_MAX_PLANS = 512


class _Plan:
    __slots__ = ("prm", "where", "address", "name", "dev", "index", "out", "parts", "state", "sizes", "spaces", "new")

    def __init__(self, name, prm, dev, out=None, parts=None, state=None, spaces=(), new=()):
        import torch
        self.prm, self.where, self.name, self.dev, self.index = prm, ctypes.addressof(prm), name, dev, dev.index
        lib, ref = load_library(), ctypes.byref(prm)
        fn = getattr(lib, name)
        self.address = ctypes.cast(fn, ctypes.c_void_p).value
        # layouts of the output like x, of one output per split, of the states, and of other new tensors
        self.out, self.parts, self.state, self.new = out, parts, state, new
        self.sizes = []
        for s in spaces:
            n = getattr(lib, s)(ref)
            if n == 0:  # parameters the library does not take: its own call says why, before it looks at a pointer
                raise SSDError(fn(ref, *[0] * (len(fn.argtypes) - 1)), name)
            self.sizes.append(n)
        self.spaces = [_layout((n,), torch.uint8, dev) for n in self.sizes]

    def call(self, *args):
        """One C call on the current stream of the tensors' device, with that device current.  Tensors that it writes come
        as they are, others as their addresses."""
        if _raw is None:
            _bind()
        if self.index == _device():
            rc = _call(self.address, self.where, *args, _raw(self.index))
        else:
            import torch
            with torch.cuda.device(self.dev):
                rc = _call(self.address, self.where, *args, _raw(self.index))
        if rc:
            raise SSDError(rc, self.name)


# torch's calls for the current device and its current stream's handle (bound at the first call)
_device = _raw = None


def _bind():
    import torch
    global _device, _raw
    torch.cuda.init()
    _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)


def _native():
    """The native module _meta (built with the library; like it, there is no fallback), its functions put in place of the
    stand-ins below."""
    global _meta, _new, _call
    load_library()
    import torch  # noqa: F401  (its libraries have to be loaded first)
    try:
        from . import _meta as m
    except ImportError as e:
        raise RuntimeError("mamba_ssd_prefill_amd._meta is not built (%s); run `python -m mamba_ssd_prefill_amd.build`"
                           % e) from e
    _meta, _new, _call = m.meta, m.new, m.call
    return m


def _meta(*tensors):
    """(key, addresses) of the tensors of a call, None for those not given."""
    return _native().meta(*tensors)


def _new(*layouts):
    """New tensors of the layouts."""
    return _native().new(*layouts)


def _call(function, *args):
    """A function of the library by its address."""
    return _native().call(function, *args)


def _layout(shape, dtype, dev):
    """What _new takes for a contiguous tensor: the key of such a one."""
    import torch
    strides, n = [], 1
    for d in reversed(shape):
        strides.append(n)
        n *= d
    head = struct.unpack("=q", _meta(torch.empty((), dtype=dtype, device=dev))[0])[0]
    return struct.pack("=%dq" % (1 + 2 * len(shape)), head | len(shape) << 32, *shape, *strides[::-1])


def _by_value(v):
    """Whether equal keys mean equal arguments: not so for a tensor, which is told apart by its identity."""
    import torch
    if isinstance(v, tuple):
        return all(_by_value(e) for e in v)
    return v is None or isinstance(v, (str, bytes, numbers.Integral, torch.dtype))


def _keep(key, plan):
    global _PLANS, _BEFORE
    if not _by_value(key):
        return plan
    if len(_PLANS) >= _MAX_PLANS // 2:
        _PLANS, _BEFORE = {}, _PLANS
    _PLANS[key] = plan
    return plan


def _older(key):
    """The plan of the older generation, if it is there."""
    plan = _BEFORE.pop(key, None)
    return plan and _keep(key, plan)


def _code(t, name):
    try:
        return _dtype_code(t)
    except KeyError:
        raise ValueError("%s must be float32, float16 or bfloat16 (got %s)" % (name, t.dtype)) from None


def _state_code(dtype):
    import torch
    codes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    if dtype not in codes:
        raise ValueError("states must be float32, float16 or bfloat16 (got %s)" % dtype)
    return codes[dtype]


def _on_gpu(t, what):
    if t.device.type != "cuda":
        raise ValueError("%s needs device tensors (got %s)" % (what, t.device))
    return t.device


def _same(dev, dtype, **tensors):
    """name=(tensor, shape) pairs: contiguous, on `dev`, of `dtype`; None passes."""
    for name, (t, shape) in tensors.items():
        if t is None:
            continue
        if tuple(t.shape) != tuple(shape):
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
        if t.device != dev:
            raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
        if t.dtype != dtype:
            raise ValueError("%s must be %s (got %s)" % (name, dtype, t.dtype))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)


def _rows(name, t, dev, dtype, shape, lead):
    """The distance between the rows of an input with one row per token ([lead..., row...]), in elements
    (0 for contiguous rows)."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    if t.dtype != dtype:
        raise ValueError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if t.is_contiguous():
        return 0
    n = 1
    for d in range(t.dim() - 1, lead - 1, -1):
        if t.shape[d] > 1 and t.stride(d) != n:
            raise ValueError("%s: the elements of a row must be contiguous" % name)
        n *= t.shape[d]
    step, count = None, 1
    for d in range(lead - 1, -1, -1):  # rows in order, a constant distance apart
        if t.shape[d] > 1:
            if step is None:
                step = t.stride(d)
            elif t.stride(d) != step * count:
                raise ValueError("%s: rows must lie a constant distance apart" % name)
            count *= t.shape[d]
    if step is None:
        return 0
    if step < n:
        raise ValueError("%s: rows overlap" % name)
    return step


def _seq(seq_idx, nseq, lead, dev):
    """The number of states: nseq with packed sequences, else the batch."""
    import torch
    if seq_idx is None:
        if nseq is not None:
            raise ValueError("nseq goes with seq_idx")
        return lead[0]
    if nseq is None or nseq < 1:
        raise ValueError("seq_idx needs nseq >= 1")
    _same(dev, torch.int32, seq_idx=(seq_idx, lead))
    return int(nseq)


def _space(workspace, dev):
    """The workspace given (the library checks its size)."""
    import torch
    if workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on %s" % dev)
    return workspace


def _states(packed, layout):
    """A new state output; entries of numbers that no sequence uses stay zero."""
    t, = _new(layout)
    return t.zero_() if packed else t


# ---- causal convolution ----------------------------------------------------------------------------
def _conv_params(x, weight, bias, activation, splits, nseq, lead):
    import torch
    dev = _on_gpu(x, "causal_conv")
    if x.dim() != len(lead) + 1:
        raise ValueError("x must have %d dimensions (got %d)" % (len(lead) + 1, x.dim()))
    code, ch = _code(x, "x"), x.shape[-1]
    if weight.dim() != 2:
        raise ValueError("weight must be [channels, width]")
    W = weight.shape[1]
    _same(dev, torch.float32, weight=(weight, (ch, W)), bias=(bias, (ch,)))
    if activation not in (None, "silu"):
        raise ValueError("activation must be None or 'silu'")
    parts = (ch,) if splits is None else tuple(int(n) for n in splits)
    if not 1 <= len(parts) <= 3 or sum(parts) != ch or min(parts) < 1:
        raise ValueError("splits must be up to three channel counts that sum to %d" % ch)
    a = parts[0]
    b = a + (parts[1] if len(parts) > 1 else 0)
    xs = _rows("x", x, dev, x.dtype, x.shape, len(lead))
    prm = ConvParams(ctypes.sizeof(ConvParams), lead[0], lead[1] if len(lead) > 1 else 1, ch, W, code,
                     1 if activation == "silu" else 0, nseq, a, b, xs)
    return prm, dev, parts


def _conv_plan(name, spaces, x, weight, bias, activation, seq_idx, nseq, splits, states, douts=()):
    lead = tuple(x.shape[:2])
    S = _seq(seq_idx, nseq, lead, x.device)
    prm, dev, parts = _conv_params(x, weight, bias, activation, splits, S, lead)
    state = (S, prm.channels, prm.width - 1)
    for n, t in states.items():
        _same(dev, x.dtype, **{n: (t, state)})
    if douts and len(douts) != len(parts):
        raise ValueError("dout must have one tensor per split")
    for d, n in zip(douts, parts):
        _same(dev, x.dtype, dout=(d, lead + (n,)))
    lay = lambda t: None if t is None else _layout(t.shape, t.dtype, dev)  # noqa: E731
    return _Plan(name, prm, dev, lay(x), [_layout(lead + (n,), x.dtype, dev) for n in parts], _layout(state, x.dtype, dev),
                 spaces, [lay(t) for t in (weight, bias) if t is not None])


def _outs(plan):
    """New outputs, one per split, and the three that the library takes."""
    outs = _new(*plan.parts)
    return outs, (*outs, None, None)[:3]


def causal_conv(x, weight, bias=None, *, activation="silu", seq_idx=None, nseq=None, initial_state=None, splits=None,
                with_final_state=True, final_state=None):
    """ssd_causal_conv: the causal depthwise convolution of x [B, L, Ch] with weight [Ch, W] float32 (W = 2, 3
    or 4), bias [Ch] and an optional SiLU (``activation`` None or "silu").  Returns (out, final_state);
    ``splits`` (up to three channel counts) makes ``out`` a tuple of contiguous tensors, e.g. the x, B and C
    of an SSD block.  States [B or nseq, Ch, W-1] hold the inputs before (after) a sequence, oldest first."""
    splits = splits if splits is None else tuple(splits)
    meta, (px, pw, pb, ps, ph, _) = _meta(x, weight, bias, seq_idx, initial_state, final_state)
    key = ("conv", meta, activation, nseq, splits)
    plan = _PLANS.get(key) or _older(key)
    if plan is None:
        plan = _keep(key, _conv_plan("ssd_causal_conv", (), x, weight, bias, activation, seq_idx, nseq, splits,
                                     dict(initial_state=initial_state, final_state=final_state)))
    outs, three = _outs(plan)
    if final_state is None and with_final_state:
        final_state = _states(seq_idx is not None, plan.state)
    plan.call(px, pw, pb, ps, ph, *three, final_state)
    return (outs[0] if splits is None else outs), final_state


def causal_conv_backward(dout, x, weight, bias=None, *, activation="silu", seq_idx=None, nseq=None, initial_state=None,
                         dfinal_state=None, splits=None, workspace=None):
    """ssd_causal_conv_backward: ConvGrads(dx, dweight, dbias, dinitial_state) of causal_conv from the gradient of
    its output (a tuple with ``splits``) and, if given, of its final state.  dbias and dinitial_state are None
    where bias and initial_state are."""
    splits = splits if splits is None else tuple(splits)
    douts = (dout,) if splits is None else tuple(dout)
    meta, (px, pw, pb, ps, ph, pf, *pd) = _meta(x, weight, bias, seq_idx, initial_state, dfinal_state, *douts)
    key = ("conv backward", meta, activation, nseq, splits)
    plan = _PLANS.get(key) or _older(key)
    if plan is None:
        plan = _keep(key, _conv_plan("ssd_causal_conv_backward", ("ssd_causal_conv_backward_workspace_size",), x, weight,
                                     bias, activation, seq_idx, nseq, splits,
                                     dict(initial_state=initial_state, dfinal_state=dfinal_state), douts))
    dx, dw, space, *db = _new(plan.out, plan.new[0], plan.spaces[0], *plan.new[1:])
    db = db[0] if db else None
    dh = None if initial_state is None else _states(seq_idx is not None, plan.state)
    workspace = space if workspace is None else _space(workspace, plan.dev)
    plan.call(*pd, *[None] * (3 - len(pd)), pf, px, pw, pb, ps, ph, dx, dw, db, dh, workspace, workspace.numel())
    return ConvGrads(dx, dw, db, dh)


def _conv_step_plan(x, weight, bias, activation, splits, state, slots):
    import torch
    lead = tuple(x.shape[:1])
    if state.dim() != 3:
        raise ValueError("state must be [nslots, channels, width - 1]")
    prm, dev, parts = _conv_params(x, weight, bias, activation, splits, state.shape[0], lead)
    _same(dev, x.dtype, state=(state, (state.shape[0], prm.channels, prm.width - 1)))
    _same(dev, torch.int32, slots=(slots, lead))
    return _Plan("ssd_causal_conv_step", prm, dev, parts=[_layout(lead + (n,), x.dtype, dev) for n in parts])


def causal_conv_step(x, weight, bias=None, *, state, activation="silu", slots=None, splits=None):
    """ssd_causal_conv_step: one token x [B, Ch] per row.  ``state`` [nslots, Ch, W-1] moves on in place; row b
    uses state ``slots[b]`` (int32; None: state b).  A row whose slot is not in [0, nslots) touches no
    state and returns zeros.  Returns out (a tuple with ``splits``)."""
    splits = splits if splits is None else tuple(splits)
    meta, (px, pw, pb, _, psl) = _meta(x, weight, bias, state, slots)
    key = ("conv step", meta, activation, splits)
    plan = _PLANS.get(key) or _older(key)
    if plan is None:
        plan = _keep(key, _conv_step_plan(x, weight, bias, activation, splits, state, slots))
    outs, three = _outs(plan)
    plan.call(px, pw, pb, state, psl, *three)
    return outs[0] if splits is None else outs


# ---- selective scan ----------------------------------------------------------------------------------
def _scan_params(x, dt, A, B, C, D, dt_bias, z, dt_softplus, state_code, nseq, lead):
    import torch
    dev = _on_gpu(x, "selective_scan")
    if x.dim() != len(lead) + 1:
        raise ValueError("x must have %d dimensions (got %d)" % (len(lead) + 1, x.dim()))
    code, ch = _code(x, "x"), x.shape[-1]
    if B.dim() != len(lead) + 2 or A.dim() != 2:
        raise ValueError("B and C must be [..., groups, dstate] and A [channels, dstate]")
    G, N = B.shape[-2:]
    _same(dev, torch.float32, A=(A, (ch, N)), D=(D, (ch,)), dt_bias=(dt_bias, (ch,)))
    rows = lambda name, t, shape: 0 if t is None else _rows(name, t, dev, x.dtype, lead + shape, len(lead))  # noqa: E731
    return ScanParams(ctypes.sizeof(ScanParams), lead[0], lead[1] if len(lead) > 1 else 1, ch, N, G, code, state_code,
                      1 if dt_softplus else 0, nseq, rows("x", x, (ch,)), rows("dt", dt, (ch,)), rows("z", z, (ch,)),
                      rows("B", B, (G, N)), rows("C", C, (G, N))), dev


def _scan_plan(name, spaces, x, dt, A, B, C, D, dt_bias, z, dt_softplus, seq_idx, nseq, state_dtype, states, like_x):
    lead = tuple(x.shape[:2])
    S = _seq(seq_idx, nseq, lead, x.device)
    if state_dtype is None:
        import torch
        given = [t for t in states.values() if t is not None]
        state_dtype = given[0].dtype if given else torch.float32
    prm, dev = _scan_params(x, dt, A, B, C, D, dt_bias, z, dt_softplus, _state_code(state_dtype), S, lead)
    state = (S, prm.channels, prm.dstate)
    for n, t in states.items():
        _same(dev, state_dtype, **{n: (t, state)})
    for n, t in like_x.items():
        _same(dev, x.dtype, **{n: (t, x.shape)})
    lay = lambda t: None if t is None else _layout(t.shape, t.dtype, dev)  # noqa: E731
    return _Plan(name, prm, dev, lay(x), state=_layout(state, state_dtype, dev), spaces=spaces,
                 new=[lay(t) for t in (x, dt, A, B, C, D, dt_bias, z)])


def selective_scan(x, dt, A, B, C, D=None, dt_bias=None, z=None, *, dt_softplus=True, seq_idx=None, nseq=None,
                   initial_state=None, state_dtype=None, save_for_backward=False, with_final_state=True,
                   final_state=None, out=None, workspace=None):
    """ssd_selective_scan over a prompt: x, dt, z [B, L, D], A [D, N] float32, B, C [B, L, G, N], D and dt_bias [D]
    float32; the rows of B and C start on multiples of 4 bytes.  Returns (out [B, L, D], final_state
    [B or nseq, D, N]), and with ``save_for_backward`` a third tensor for selective_scan_backward, N / 4 times as large as a
    16-bit x.
    ``state_dtype`` defaults to initial_state's, else float32."""
    meta, (px, pdt, pA, pB, pC, pD, pb, pz, ps, ph, _, _) = _meta(x, dt, A, B, C, D, dt_bias, z, seq_idx, initial_state,
                                                                  final_state, out)
    key = ("scan", meta, dt_softplus, nseq, state_dtype)
    plan = _PLANS.get(key) or _older(key)
    if plan is None:
        plan = _keep(key, _scan_plan("ssd_selective_scan", ("ssd_selective_scan_workspace_size",
                                                            "ssd_selective_scan_saved_size"),
                                     x, dt, A, B, C, D, dt_bias, z, dt_softplus, seq_idx, nseq, state_dtype,
                                     dict(initial_state=initial_state, final_state=final_state), dict(out=out)))
    if out is None:
        out, = _new(plan.out)
    if final_state is None and with_final_state:
        final_state = _states(seq_idx is not None, plan.state)
    workspace = _new(plan.spaces[0])[0] if workspace is None else _space(workspace, plan.dev)
    saved = _new(plan.spaces[1])[0] if save_for_backward else None
    plan.call(px, pdt, pA, pB, pC, pD, pb, pz, ps, ph, out, final_state, saved, workspace, workspace.numel())
    return (out, final_state, saved) if save_for_backward else (out, final_state)


def selective_scan_backward(dout, x, dt, A, B, C, D=None, dt_bias=None, z=None, *, saved, dt_softplus=True, seq_idx=None,
                            nseq=None, initial_state=None, dfinal_state=None, state_dtype=None, workspace=None):
    """ssd_selective_scan_backward: ScanGrads of selective_scan from dout [B, L, D], dfinal_state (None: zeros), the
    forward's inputs and the ``saved`` tensor it returned.  ddt is the gradient of the raw dt.  dD, ddt_bias,
    dz and dinitial_state are None where the input is."""
    import torch
    meta, (pg, px, pdt, pA, pB, pC, pD, pb, pz, ps, ph, pf, psv) = _meta(dout, x, dt, A, B, C, D, dt_bias, z, seq_idx,
                                                                         initial_state, dfinal_state, saved)
    key = ("scan backward", meta, dt_softplus, nseq, state_dtype)
    plan = _PLANS.get(key) or _older(key)
    if plan is None:
        plan = _scan_plan("ssd_selective_scan_backward", ("ssd_selective_scan_backward_workspace_size",
                                                          "ssd_selective_scan_saved_size"),
                          x, dt, A, B, C, D, dt_bias, z, dt_softplus, seq_idx, nseq, state_dtype,
                          dict(initial_state=initial_state, dfinal_state=dfinal_state), dict(dout=dout))
        _same(plan.dev, torch.uint8, saved=(saved, (plan.sizes[1],)))
        _keep(key, plan)
    made = iter(_new(*[n for n in plan.new if n is not None]))
    g = ScanGrads(*[None if n is None else next(made) for n in plan.new],
                  None if initial_state is None else _states(seq_idx is not None, plan.state))
    workspace = _new(plan.spaces[0])[0] if workspace is None else _space(workspace, plan.dev)
    plan.call(pg, pf, px, pdt, pA, pB, pC, pD, pb, pz, ps, ph, psv, *g, workspace, workspace.numel())
    return g


def _scan_step_plan(x, dt, A, B, C, D, dt_bias, z, state, slots, dt_softplus, out):
    import torch
    lead = tuple(x.shape[:1])
    if state.dim() != 3:
        raise ValueError("state must be [nslots, channels, dstate]")
    prm, dev = _scan_params(x, dt, A, B, C, D, dt_bias, z, dt_softplus, _state_code(state.dtype), state.shape[0], lead)
    _same(dev, state.dtype, state=(state, (state.shape[0], prm.channels, prm.dstate)))
    _same(dev, torch.int32, slots=(slots, lead))
    _same(dev, x.dtype, out=(out, x.shape))
    return _Plan("ssd_selective_scan_step", prm, dev, _layout(x.shape, x.dtype, dev))


def selective_scan_step(x, dt, A, B, C, D=None, dt_bias=None, z=None, *, state, slots=None, dt_softplus=True, out=None):
    """ssd_selective_scan_step: one token per row; x, dt, z [B, D], B, C [B, G, N].  ``state`` [nslots, D, N] is
    updated in place; row b uses state ``slots[b]`` (int32; None: state b).  A row whose slot is not in
    [0, nslots) touches no state and returns zeros.  Returns out [B, D]."""
    meta, (px, pdt, pA, pB, pC, pD, pb, pz, _, psl, _) = _meta(x, dt, A, B, C, D, dt_bias, z, state, slots, out)
    key = ("scan step", meta, dt_softplus)
    plan = _PLANS.get(key) or _older(key)
    if plan is None:
        plan = _keep(key, _scan_step_plan(x, dt, A, B, C, D, dt_bias, z, state, slots, dt_softplus, out))
    if out is None:
        out, = _new(plan.out)
    plan.call(px, pdt, pA, pB, pC, pD, pb, pz, state, psl, out)
    return out


# ---- 8-bit state cache ---------------------------------------------------------------------------------
def state_cache(nslots, shape, *, group=64, format="int8", device="cuda"):
    """An empty pool for nslots states of ``shape``: codes [nslots, *shape] (torch.int8, or torch.float8_e4m3fn
    for format "e4m3") and scales [nslots, values / group] float32.  ``group`` is 16, 32, 64 or 128."""
    import torch
    if format not in ("int8", "e4m3"):
        raise ValueError("format must be 'int8' or 'e4m3'")
    n = 1
    for d in shape:
        n *= int(d)
    if group not in (16, 32, 64, 128) or n < 1 or n % group:
        raise ValueError("group must be 16, 32, 64 or 128 and divide the %d values of a state" % n)
    code = torch.int8 if format == "int8" else torch.float8_e4m3fn
    codes = torch.zeros((nslots, n), dtype=torch.int8, device=device).view(code).view((nslots,) + tuple(shape))
    return codes, torch.zeros((nslots, n // group), dtype=torch.float32, device=device)


def _cache_plan(name, codes, scales, slots, batch, state_dtype, state):
    import torch
    dev = _on_gpu(codes, "the state cache")
    formats = {torch.int8: CACHE_INT8, torch.float8_e4m3fn: CACHE_E4M3}
    if codes.dtype not in formats:
        raise ValueError("codes must be int8 or float8_e4m3fn (got %s)" % codes.dtype)
    nslots, elems = codes.shape[0], codes[0].numel() if codes.shape[0] else 0
    if scales.dim() != 2 or scales.shape[0] != nslots or not scales.shape[1] or elems % scales.shape[1]:
        raise ValueError("scales must be [nslots, values / group]")
    shape = (batch,) + tuple(codes.shape[1:])
    _same(dev, codes.dtype, codes=(codes, codes.shape))
    _same(dev, torch.float32, scales=(scales, scales.shape))
    _same(dev, torch.int32, slots=(slots, (batch,)))
    _same(dev, state_dtype, state=(state, shape))
    prm = CacheParams(ctypes.sizeof(CacheParams), batch, nslots, elems, elems // scales.shape[1], formats[codes.dtype],
                      _state_code(state_dtype))
    return _Plan(name, prm, dev, _layout(shape, state_dtype, dev))


def state_cache_write(state, codes, scales, slots=None):
    """ssd_state_cache_write: state [B, ...] (float32, float16 or bfloat16) into the slots ``slots[b]`` (int32;
    None: b) of a pool made by state_cache.  Rows whose slot is not in [0, nslots) are skipped."""
    meta, (ps, _, _, psl) = _meta(state, codes, scales, slots)
    key = ("cache write", meta)
    plan = _PLANS.get(key) or _older(key)
    if plan is None:
        plan = _keep(key, _cache_plan("ssd_state_cache_write", codes, scales, slots, state.shape[0], state.dtype, state))
    plan.call(ps, psl, codes, scales)


def state_cache_read(codes, scales, slots=None, *, state_dtype=None, out=None):
    """ssd_state_cache_read: the states of ``slots`` (int32 [B]; None: every slot), in ``state_dtype`` (default
    float32) or into ``out`` [B, ...].  A row whose slot is not in [0, nslots) reads a zero state."""
    import torch
    meta, (pc, psc, psl, _) = _meta(codes, scales, slots, out)
    key = ("cache read", meta, state_dtype)
    plan = _PLANS.get(key) or _older(key)
    if plan is None:
        batch = codes.shape[0] if slots is None and out is None else (out if slots is None else slots).shape[0]
        if state_dtype is None:
            state_dtype = torch.float32 if out is None else out.dtype
        plan = _keep(key, _cache_plan("ssd_state_cache_read", codes, scales, slots, batch, state_dtype, out))
    if out is None:
        out, = _new(plan.out)
    plan.call(pc, psc, psl, out)
    return out
