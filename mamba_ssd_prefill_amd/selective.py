"""The selective state space scan, its short causal convolution and the 8-bit state cache.

A thin ctypes binding over the second half of include/mamba_ssd.h, in the manner of the package's
other entry points: it checks arguments, allocates outputs and workspaces, and passes pointers and
the current stream of the tensors' device.  The names are re-exported by the package:

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
such as the halves of a joint projection; everything else is contiguous.  Sequences packed into a
batch row are told apart by ``seq_idx`` (int32 [B, L], numbers in [0, nseq); -1: padding), and
states then have one entry per number instead of one per batch row.
"""
import collections
import ctypes

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
def _p(t):
    return None if t is None else t.data_ptr()


def _call(name, prm, dev, *args):
    """One C call on the current stream of `dev`, with that device current."""
    import torch
    fn = getattr(load_library(), name)
    if dev.index is None or dev.index == torch.cuda.current_device():
        rc = fn(ctypes.byref(prm), *args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(ctypes.byref(prm), *args, torch.cuda.current_stream(dev).cuda_stream)
    if rc:
        raise SSDError(rc, name)


def _size(name, prm):
    """A size the library asks for; its functions give 0 for parameters they do not take."""
    n = getattr(load_library(), name)(ctypes.byref(prm))
    if n == 0:
        raise SSDError(3, name)
    return n


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


def _workspace(workspace, n, dev):
    import torch
    if workspace is None:
        return torch.empty(n, dtype=torch.uint8, device=dev)
    if workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on %s" % dev)
    return workspace


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


def _three(ts):
    return [_p(t) for t in ts] + [None] * (3 - len(ts))


def causal_conv(x, weight, bias=None, *, activation="silu", seq_idx=None, nseq=None, initial_state=None, splits=None,
                with_final_state=True, final_state=None):
    """ssd_causal_conv: the causal depthwise convolution of x [B, L, Ch] with weight [Ch, W] float32 (W = 2, 3
    or 4), bias [Ch] and an optional SiLU (``activation`` None or "silu").  Returns (out, final_state);
    ``splits`` (up to three channel counts) makes ``out`` a tuple of contiguous tensors, e.g. the x, B and C
    of an SSD block.  States [B or nseq, Ch, W-1] hold the inputs before (after) a sequence, oldest first."""
    import torch
    lead = tuple(x.shape[:2])
    S = _seq(seq_idx, nseq, lead, x.device)
    prm, dev, parts = _conv_params(x, weight, bias, activation, splits, S, lead)
    shape = (S, prm.channels, prm.width - 1)
    _same(dev, x.dtype, initial_state=(initial_state, shape), final_state=(final_state, shape))
    outs = tuple(torch.empty(lead + (n,), dtype=x.dtype, device=dev) for n in parts)
    if final_state is None and with_final_state:
        # numbers that no sequence uses keep their entry
        final_state = (torch.empty if seq_idx is None else torch.zeros)(shape, dtype=x.dtype, device=dev)
    _call("ssd_causal_conv", prm, dev, _p(x), _p(weight), _p(bias), _p(seq_idx), _p(initial_state), *_three(outs),
          _p(final_state))
    return (outs[0] if splits is None else outs), final_state


def causal_conv_backward(dout, x, weight, bias=None, *, activation="silu", seq_idx=None, nseq=None, initial_state=None,
                         dfinal_state=None, splits=None, workspace=None):
    """ssd_causal_conv_backward: ConvGrads(dx, dweight, dbias, dinitial_state) of causal_conv from the gradient of
    its output (a tuple with ``splits``) and, if given, of its final state.  dbias and dinitial_state are None
    where bias and initial_state are."""
    import torch
    lead = tuple(x.shape[:2])
    S = _seq(seq_idx, nseq, lead, x.device)
    prm, dev, parts = _conv_params(x, weight, bias, activation, splits, S, lead)
    shape = (S, prm.channels, prm.width - 1)
    douts = (dout,) if splits is None else tuple(dout)
    if len(douts) != len(parts):
        raise ValueError("dout must have one tensor per split")
    for d, n in zip(douts, parts):
        _same(dev, x.dtype, dout=(d, lead + (n,)))
    _same(dev, x.dtype, initial_state=(initial_state, shape), dfinal_state=(dfinal_state, shape))
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    dw = torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    dh = None
    if initial_state is not None:
        dh = (torch.empty if seq_idx is None else torch.zeros)(shape, dtype=x.dtype, device=dev)
    workspace = _workspace(workspace, _size("ssd_causal_conv_backward_workspace_size", prm), dev)
    _call("ssd_causal_conv_backward", prm, dev, *_three(douts), _p(dfinal_state), _p(x), _p(weight), _p(bias),
          _p(seq_idx), _p(initial_state), _p(dx), _p(dw), _p(db), _p(dh), _p(workspace), workspace.numel())
    return ConvGrads(dx, dw, db, dh)


def causal_conv_step(x, weight, bias=None, *, state, activation="silu", slots=None, splits=None):
    """ssd_causal_conv_step: one token x [B, Ch] per row.  ``state`` [nslots, Ch, W-1] moves on in place; row b
    uses state ``slots[b]`` (int32; None: state b).  A row whose slot is not in [0, nslots) touches no
    state and returns zeros.  Returns out (a tuple with ``splits``)."""
    import torch
    lead = tuple(x.shape[:1])
    if state.dim() != 3:
        raise ValueError("state must be [nslots, channels, width - 1]")
    prm, dev, parts = _conv_params(x, weight, bias, activation, splits, state.shape[0], lead)
    _same(dev, x.dtype, state=(state, (state.shape[0], prm.channels, prm.width - 1)))
    _same(dev, torch.int32, slots=(slots, lead))
    outs = tuple(torch.empty(lead + (n,), dtype=x.dtype, device=dev) for n in parts)
    _call("ssd_causal_conv_step", prm, dev, _p(x), _p(weight), _p(bias), _p(state), _p(slots), *_three(outs))
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


def selective_scan(x, dt, A, B, C, D=None, dt_bias=None, z=None, *, dt_softplus=True, seq_idx=None, nseq=None,
                   initial_state=None, state_dtype=None, save_for_backward=False, with_final_state=True,
                   final_state=None, out=None, workspace=None):
    """ssd_selective_scan over a prompt: x, dt, z [B, L, D], A [D, N] float32, B, C [B, L, G, N], D and dt_bias [D]
    float32.  Returns (out [B, L, D], final_state [B or nseq, D, N]), and with ``save_for_backward`` a third
    tensor for selective_scan_backward.  ``state_dtype`` defaults to initial_state's, else float32."""
    import torch
    lead = tuple(x.shape[:2])
    S = _seq(seq_idx, nseq, lead, x.device)
    if state_dtype is None:
        state_dtype = initial_state.dtype if initial_state is not None else torch.float32
    prm, dev = _scan_params(x, dt, A, B, C, D, dt_bias, z, dt_softplus, _state_code(state_dtype), S, lead)
    shape = (S, prm.channels, prm.dstate)
    _same(dev, state_dtype, initial_state=(initial_state, shape), final_state=(final_state, shape))
    _same(dev, x.dtype, out=(out, x.shape))
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    if final_state is None and with_final_state:
        final_state = (torch.empty if seq_idx is None else torch.zeros)(shape, dtype=state_dtype, device=dev)
    workspace = _workspace(workspace, _size("ssd_selective_scan_workspace_size", prm), dev)
    saved = None
    if save_for_backward:
        saved = torch.empty(_size("ssd_selective_scan_saved_size", prm), dtype=torch.uint8, device=dev)
    _call("ssd_selective_scan", prm, dev, _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(dt_bias), _p(z), _p(seq_idx),
          _p(initial_state), _p(out), _p(final_state), _p(saved), _p(workspace), workspace.numel())
    return (out, final_state, saved) if save_for_backward else (out, final_state)


def selective_scan_backward(dout, x, dt, A, B, C, D=None, dt_bias=None, z=None, *, saved, dt_softplus=True, seq_idx=None,
                            nseq=None, initial_state=None, dfinal_state=None, state_dtype=None, workspace=None):
    """ssd_selective_scan_backward: ScanGrads of selective_scan from dout [B, L, D], dfinal_state (None: zeros), the
    forward's inputs and the ``saved`` tensor it returned.  ddt is the gradient of the raw dt.  dD, ddt_bias,
    dz and dinitial_state are None where the input is."""
    import torch
    lead = tuple(x.shape[:2])
    S = _seq(seq_idx, nseq, lead, x.device)
    if state_dtype is None:
        given = [t for t in (initial_state, dfinal_state) if t is not None]
        state_dtype = given[0].dtype if given else torch.float32
    prm, dev = _scan_params(x, dt, A, B, C, D, dt_bias, z, dt_softplus, _state_code(state_dtype), S, lead)
    shape = (S, prm.channels, prm.dstate)
    _same(dev, state_dtype, initial_state=(initial_state, shape), dfinal_state=(dfinal_state, shape))
    _same(dev, x.dtype, dout=(dout, x.shape))
    _same(dev, torch.uint8, saved=(saved, (_size("ssd_selective_scan_saved_size", prm),)))
    like = lambda t: None if t is None else torch.empty(t.shape, dtype=t.dtype, device=dev)  # noqa: E731
    g = ScanGrads(like(x), like(dt), like(A), like(B), like(C), like(D), like(dt_bias), like(z),
                  None if initial_state is None else
                  (torch.empty if seq_idx is None else torch.zeros)(shape, dtype=state_dtype, device=dev))
    workspace = _workspace(workspace, _size("ssd_selective_scan_backward_workspace_size", prm), dev)
    _call("ssd_selective_scan_backward", prm, dev, _p(dout), _p(dfinal_state), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D),
          _p(dt_bias), _p(z), _p(seq_idx), _p(initial_state), _p(saved), _p(g.dx), _p(g.ddt), _p(g.dA), _p(g.dB),
          _p(g.dC), _p(g.dD), _p(g.ddt_bias), _p(g.dz), _p(g.dinitial_state), _p(workspace), workspace.numel())
    return g


def selective_scan_step(x, dt, A, B, C, D=None, dt_bias=None, z=None, *, state, slots=None, dt_softplus=True, out=None):
    """ssd_selective_scan_step: one token per row; x, dt, z [B, D], B, C [B, G, N].  ``state`` [nslots, D, N] is
    updated in place; row b uses state ``slots[b]`` (int32; None: state b).  A row whose slot is not in
    [0, nslots) touches no state and returns zeros.  Returns out [B, D]."""
    import torch
    lead = tuple(x.shape[:1])
    if state.dim() != 3:
        raise ValueError("state must be [nslots, channels, dstate]")
    prm, dev = _scan_params(x, dt, A, B, C, D, dt_bias, z, dt_softplus, _state_code(state.dtype), state.shape[0], lead)
    _same(dev, state.dtype, state=(state, (state.shape[0], prm.channels, prm.dstate)))
    _same(dev, torch.int32, slots=(slots, lead))
    _same(dev, x.dtype, out=(out, x.shape))
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    _call("ssd_selective_scan_step", prm, dev, _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(dt_bias), _p(z), _p(state),
          _p(slots), _p(out))
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


def _cache_params(codes, scales, slots, batch, state_code):
    import torch
    dev = _on_gpu(codes, "the state cache")
    formats = {torch.int8: CACHE_INT8, torch.float8_e4m3fn: CACHE_E4M3}
    if codes.dtype not in formats:
        raise ValueError("codes must be int8 or float8_e4m3fn (got %s)" % codes.dtype)
    nslots, elems = codes.shape[0], codes[0].numel() if codes.shape[0] else 0
    if scales.dim() != 2 or scales.shape[0] != nslots or not scales.shape[1] or elems % scales.shape[1]:
        raise ValueError("scales must be [nslots, values / group]")
    _same(dev, codes.dtype, codes=(codes, codes.shape))
    _same(dev, torch.float32, scales=(scales, scales.shape))
    _same(dev, torch.int32, slots=(slots, (batch,)))
    return CacheParams(ctypes.sizeof(CacheParams), batch, nslots, elems, elems // scales.shape[1], formats[codes.dtype],
                       state_code), dev


def state_cache_write(state, codes, scales, slots=None):
    """ssd_state_cache_write: state [B, ...] (float32, float16 or bfloat16) into the slots ``slots[b]`` (int32;
    None: b) of a pool made by state_cache.  Rows whose slot is not in [0, nslots) are skipped."""
    prm, dev = _cache_params(codes, scales, slots, state.shape[0], _state_code(state.dtype))
    _same(dev, state.dtype, state=(state, (state.shape[0],) + tuple(codes.shape[1:])))
    _call("ssd_state_cache_write", prm, dev, _p(state), _p(slots), _p(codes), _p(scales))


def state_cache_read(codes, scales, slots=None, *, state_dtype=None, out=None):
    """ssd_state_cache_read: the states of ``slots`` (int32 [B]; None: every slot), in ``state_dtype`` (default
    float32) or into ``out`` [B, ...].  A row whose slot is not in [0, nslots) reads a zero state."""
    import torch
    batch = codes.shape[0] if slots is None and out is None else (out if slots is None else slots).shape[0]
    if state_dtype is None:
        state_dtype = torch.float32 if out is None else out.dtype
    prm, dev = _cache_params(codes, scales, slots, batch, _state_code(state_dtype))
    shape = (batch,) + tuple(codes.shape[1:])
    _same(dev, state_dtype, out=(out, shape))
    if out is None:
        out = torch.empty(shape, dtype=state_dtype, device=dev)
    _call("ssd_state_cache_read", prm, dev, _p(codes), _p(scales), _p(slots), _p(out))
    return out
