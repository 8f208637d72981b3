"""Refusals of the residual norm, the matrix product and the gated recurrence, without a GPU: every C call here
fails exactly one host check (fake aligned addresses), so nothing is launched; and the binding's structs have the
header's layout."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import mamba_ssd_prefill_amd as ssd
from mamba_ssd_prefill_amd import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULLP, SHAPE, UNSUP, MISAL, WS_SMALL, HIP, TIMEOUT, BADARG = range(9)
FAKE = 1 << 44  # apart, so that only overlaps made on purpose are overlaps


@pytest.fixture(scope="module")
def lib():
    return ssd.load_library()


def norm_prm(**kw):
    p = dict(rows=30, width=64, in_dtype=2, sum_dtype=2, format=-1, eps=1e-5, x_stride=0, residual_stride=0)
    p.update(kw)
    return ssd.NormParams(ctypes.sizeof(ssd.NormParams), *p.values())


def linear_prm(**kw):
    p = dict(rows=30, width=64, outs=96, in_dtype=2, out_dtype=2, act=0, x_stride=0, residual_stride=0)
    p.update(kw)
    return ssd.LinearParams(ctypes.sizeof(ssd.LinearParams), *p.values())


def rec_prm(**kw):
    p = dict(batch=2, seqlen=30, channels=64, in_dtype=2, state_dtype=0, normalize=1, nseq=0, x_stride=0, gate_stride=0,
             in_stride=0)
    p.update(kw)
    return ssd.RecurrenceParams(ctypes.sizeof(ssd.RecurrenceParams), *p.values())


# the pointer arguments of each entry point, those that may be NULL in the calls below, and those left out in them
ARGS = {
    "ssd_rms_norm": ("x w residual out scales sum", "residual", "scales"),
    "ssd_rms_norm_backward": ("dout s w dsum dx dres dw ws", "dsum dx dres dw", ""),
    "ssd_linear": ("x w bias res sx sw pre out ws", "bias res sx sw pre", "sx sw"),
    "ssd_linear_backward": ("dout x w pre dx dw db ws", "pre dx dw db", "pre"),
    "ssd_gated_recurrence": ("x gate A ig gb ib seq h0 out fin saved ws", "ig gb ib seq h0 fin saved", "seq"),
    "ssd_gated_recurrence_backward": ("dout dfin x gate A ig gb ib seq h0 saved dx dgate dA dig dgb dib dh0 ws",
                                      "dfin ig gb ib seq h0 dgb dib dh0", "seq"),
    "ssd_gated_recurrence_step": ("x gate A ig gb ib state slots out", "ig gb ib slots", "slots"),
}
PRM = {"ssd_rms": norm_prm, "ssd_lin": linear_prm, "ssd_gat": rec_prm}


def params_for(name, **kw):
    if name.endswith("_step"):
        kw = dict(dict(seqlen=1, nseq=2), **kw)
    return PRM[name[:7]](**kw)


def call(lib, name, prm, ws_bytes=1 << 40, **over):
    fields, _, without = (s.split() for s in ARGS[name])
    vals = {f: None if f in without else FAKE + (i << 41) for i, f in enumerate(fields)}
    vals.update(over)
    a = [vals[f] for f in fields]
    if "ws" in fields:
        a.append(ws_bytes)
    return getattr(lib, name)(ctypes.byref(prm) if prm is not None else None, *a, None)


@pytest.mark.parametrize("name", sorted(ARGS))
def test_null_pointers(lib, name):
    assert call(lib, name, None) == NULLP
    fields, free, _ = (s.split() for s in ARGS[name])
    for f in fields:
        if f not in free and f not in ("scales",):
            assert call(lib, name, params_for(name), **{f: None}) == NULLP, f
    if name == "ssd_rms_norm":
        assert call(lib, name, norm_prm(format=0)) == NULLP                       # codes need their scales
        assert call(lib, name, norm_prm(), scales=FAKE) == BADARG                 # and values have none
        assert call(lib, name, norm_prm(), residual=None) == BADARG               # a sum without a residual
    if name == "ssd_rms_norm_backward":
        assert call(lib, name, norm_prm(), dx=None, dres=None) == NULLP
    if name == "ssd_linear":
        assert call(lib, name, linear_prm(), sx=FAKE) == BADARG
        assert call(lib, name, linear_prm(), sw=FAKE) == BADARG
    if name == "ssd_linear_backward":
        assert call(lib, name, linear_prm(), dx=None, dw=None, db=None) == NULLP
        assert call(lib, name, linear_prm(act=1)) == NULLP                        # pre is needed
        assert call(lib, name, linear_prm(), pre=FAKE) == BADARG
    if name.startswith("ssd_gated"):
        assert call(lib, name, params_for(name), ig=None) == BADARG               # in_bias without in_gate
    if name == "ssd_gated_recurrence_backward":
        assert call(lib, name, rec_prm(), dig=None) == NULLP
        assert call(lib, name, rec_prm(), ig=None, ib=None, dib=None) == BADARG   # its gradient without in_gate
        assert call(lib, name, rec_prm(), ig=None, ib=None, dig=None) == BADARG


FP32 = {"ssd_rms_norm": ("w",), "ssd_rms_norm_backward": ("w", "dw"), "ssd_linear": ("bias",), "ssd_linear_backward": ("db",),
        "ssd_gated_recurrence": ("A", "gb", "ib", "saved", "h0", "fin"),
        "ssd_gated_recurrence_backward": ("A", "gb", "ib", "saved", "h0", "dfin", "dA", "dgb", "dib", "dh0"),
        "ssd_gated_recurrence_step": ("A", "gb", "ib", "state")}
WIDE = {"ssd_linear": ("x", "w"), "ssd_linear_backward": ("dout",)}


@pytest.mark.parametrize("name", sorted(ARGS))
def test_misaligned(lib, name):
    for i, f in enumerate(ARGS[name][0].split()):
        a = 256 if f == "ws" else 16 if f in WIDE.get(name, ()) else 4 if f in FP32[name] else 2
        kw, p = {}, {}
        if f in ("scales",):
            a, p = 4, dict(format=1)
        if f in ("sx", "sw"):
            a, p = 4, dict(in_dtype=3)
        if f in ("seq", "slots"):
            a, p = 4, dict(nseq=2)
        if f == "pre" and name == "ssd_linear_backward":
            p = dict(act=1)
        if f == "out" and p.get("format"):
            continue
        kw[f] = FAKE + (i << 41) + a // 2
        assert call(lib, name, params_for(name, **p), **kw) == MISAL, (f, a)
    if name == "ssd_linear_backward":  # dout itself is an operand only without an activation, of whole pieces, for dx
        for prm, kw in ((linear_prm(act=1), dict(pre=FAKE)), (linear_prm(outs=97), {}), (linear_prm(), dict(dx=None))):
            assert call(lib, name, prm, dout=FAKE + 2, ws_bytes=0, **kw) == WS_SMALL
            assert call(lib, name, prm, dout=FAKE + 1, ws_bytes=0, **kw) == MISAL
    if name == "ssd_linear":  # the rows of a view may start anywhere, by their elements
        assert call(lib, name, linear_prm(x_stride=70), x=FAKE + 2, ws_bytes=0) == WS_SMALL
        assert call(lib, name, linear_prm(x_stride=70), x=FAKE + 1) == MISAL


@pytest.mark.parametrize("dtype,es", [(0, 4), (1, 2), (2, 2), (3, 1), (4, 1)])
@pytest.mark.parametrize("rows", [1, 30, 4000])
def test_rows_cut_out_of_a_joint_weight(lib, dtype, es, rows):
    """A weight that starts k rows behind an aligned one's first row is taken, whatever the rows' length."""
    for width in (64, 63, 65, 66, 68, 72, 1, 2, 2561, 2562):
        row = width * es
        prm = linear_prm(in_dtype=dtype, rows=rows, width=width)
        for k in (1, 2, 3, 7):
            assert call(lib, "ssd_linear", prm, w=FAKE + k * row, ws_bytes=0) == WS_SMALL, (width, k)
        need = 16 if row % 16 == 0 else 4 if row % 4 == 0 else es
        if need > 1:
            assert call(lib, "ssd_linear", prm, w=FAKE + need // 2) == MISAL, width


@pytest.mark.parametrize("dtype,es", [(0, 4), (1, 2), (2, 2), (3, 1), (4, 1)])
@pytest.mark.parametrize("rows", [1, 30])
def test_contiguous_rows_that_start_anywhere(lib, dtype, es, rows):
    """One row of a view counts as contiguous, and so do rows behind an odd offset: with their stride given they are taken as a
    view's are, and the workspace has room to copy them."""
    prm, size = linear_prm(in_dtype=dtype, rows=rows, x_stride=64), lib.ssd_linear_workspace_size
    assert call(lib, "ssd_linear", prm, x=FAKE + es, ws_bytes=0) == WS_SMALL
    if es > 1:
        assert call(lib, "ssd_linear", prm, x=FAKE + es // 2) == MISAL
    room = size(ctypes.byref(prm)) - size(ctypes.byref(linear_prm(in_dtype=dtype, rows=rows)))
    assert room >= rows * 64 * es - 256  # (a product without copies has one region of 256 bytes)


@pytest.mark.parametrize("name", ["ssd_rms_norm", "ssd_rms_norm_backward"])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(width=0), SHAPE), (dict(width=16385), UNSUP),
    (dict(in_dtype=3), BADARG), (dict(in_dtype=-1), BADARG), (dict(sum_dtype=1), BADARG), (dict(format=2), BADARG),
    (dict(format=-2), BADARG), (dict(eps=-1e-9), BADARG), (dict(eps=float("nan")), BADARG), (dict(eps=float("inf")), BADARG),
    (dict(x_stride=63), SHAPE), (dict(x_stride=-64), SHAPE), (dict(x_stride=1 << 31), SHAPE), (dict(residual_stride=1), SHAPE)])
def test_norm_parameters(lib, name, kw, code):
    assert call(lib, name, norm_prm(**kw)) == code


def test_norm_backward_has_no_codes(lib):
    assert call(lib, "ssd_rms_norm_backward", norm_prm(format=0)) == BADARG


@pytest.mark.parametrize("name", ["ssd_linear", "ssd_linear_backward"])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), SHAPE), (dict(width=0), SHAPE), (dict(outs=0), SHAPE), (dict(in_dtype=5), BADARG), (dict(in_dtype=-1), BADARG),
    (dict(out_dtype=3), BADARG), (dict(act=3), BADARG), (dict(act=-1), BADARG), (dict(x_stride=63), SHAPE),
    (dict(x_stride=1 << 31), SHAPE), (dict(residual_stride=95), SHAPE), (dict(width=1 << 21), SHAPE),
    (dict(rows=2**31 - 1, outs=2**31 - 1), SHAPE), (dict(rows=2**31 - 1, width=1 << 18), SHAPE),
    (dict(outs=2**31 - 1, width=1 << 18), SHAPE), (dict(rows=1 << 19, outs=1 << 19, width=1 << 16), SHAPE)])
def test_linear_parameters(lib, name, kw, code):
    assert call(lib, name, linear_prm(**kw)) == code


def test_linear_codes(lib):
    assert call(lib, "ssd_linear", linear_prm(in_dtype=3, width=131072)) == UNSUP  # -128 * -128 * K would pass 2^31 - 1
    assert call(lib, "ssd_linear", linear_prm(in_dtype=3, width=131071), ws_bytes=0) == WS_SMALL
    for t in (3, 4):
        assert call(lib, "ssd_linear_backward", linear_prm(in_dtype=t, out_dtype=0)) == BADARG
    assert call(lib, "ssd_linear_backward", linear_prm(out_dtype=0)) == BADARG
    # contractions of the gradients: rows and outs
    assert call(lib, "ssd_linear_backward", linear_prm(rows=1 << 21)) == SHAPE
    assert call(lib, "ssd_linear_backward", linear_prm(outs=1 << 21)) == SHAPE


@pytest.mark.parametrize("name", ["ssd_gated_recurrence", "ssd_gated_recurrence_backward", "ssd_gated_recurrence_step"])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), SHAPE), (dict(channels=0), SHAPE), (dict(seqlen=0), SHAPE), (dict(channels=1 << 21), SHAPE),
    (dict(in_dtype=3), BADARG), (dict(state_dtype=-1), BADARG), (dict(normalize=2), BADARG), (dict(x_stride=63), SHAPE),
    (dict(gate_stride=-1), SHAPE), (dict(in_stride=1), SHAPE), (dict(x_stride=1 << 31), SHAPE),
    (dict(batch=1 << 20, seqlen=1 << 12), SHAPE)])
def test_recurrence_parameters(lib, name, kw, code):
    if name.endswith("_step") and kw.get("seqlen"):
        kw = dict(seqlen=2)
    assert call(lib, name, params_for(name, **kw)) == code


@pytest.mark.parametrize("name", ["ssd_gated_recurrence", "ssd_gated_recurrence_backward"])
def test_recurrence_sizes_past_a_tile_s_offsets(lib, name):
    for f in ("x_stride", "gate_stride", "in_stride"):
        assert call(lib, name, rec_prm(**{f: 1 << 21})) == SHAPE
        assert call(lib, name, rec_prm(**{f: (1 << 21) - 1}), ws_bytes=0) == WS_SMALL
        assert call(lib, "ssd_gated_recurrence_step", params_for("ssd_gated_recurrence_step", **{f: 1 << 21}), slots=FAKE + 2) == MISAL
    # workgroups of 256 lanes: one for 64 tokens and 128 bytes of channels
    for t, ch in ((0, 32), (1, 64), (2, 64)):
        assert call(lib, name, rec_prm(batch=1, seqlen=(1 << 30) - 64, channels=ch, in_dtype=t), ws_bytes=0) == WS_SMALL
        assert call(lib, name, rec_prm(batch=1, seqlen=(1 << 30) - 63, channels=1, in_dtype=t)) == SHAPE
        assert call(lib, name, rec_prm(batch=1, seqlen=1 << 29, channels=ch + 1, in_dtype=t)) == SHAPE


def test_recurrence_step_lanes(lib):
    name = "ssd_gated_recurrence_step"
    assert call(lib, name, params_for(name, batch=1 << 14, channels=1 << 18, nseq=1 << 14)) == SHAPE


@pytest.mark.parametrize("name", sorted(ARGS))
def test_short_struct(lib, name):
    prm = params_for(name)
    prm.struct_size -= 1
    assert call(lib, name, prm) == BADARG


def test_packed_input_and_pools_need_their_number_of_states(lib):
    assert call(lib, "ssd_gated_recurrence", rec_prm(), seq=FAKE) == SHAPE
    assert call(lib, "ssd_gated_recurrence_backward", rec_prm(), seq=FAKE) == SHAPE
    step = "ssd_gated_recurrence_step"
    assert call(lib, step, params_for(step, nseq=0)) == SHAPE
    assert call(lib, step, params_for(step, nseq=3)) == SHAPE  # no slots: one state a row


def test_overlaps_are_refused(lib):
    """Outputs over inputs that other lanes or workgroups still read; the sum over the residual in place is none."""
    def norm(prm, **kw):
        return call(lib, "ssd_rms_norm", prm, **kw)
    n = 30 * 64 * 2
    for shift in (2, -2, n - 2, 2 - n):
        assert norm(norm_prm(), residual=FAKE, sum=FAKE + shift) == BADARG
    assert norm(norm_prm(residual_stride=70), residual=FAKE, sum=FAKE) == BADARG
    # (refused behind these checks only by another one: nothing is launched)
    assert norm(norm_prm(residual_stride=64), residual=FAKE, sum=FAKE, x=FAKE + 1) == MISAL
    m = 30 * 96 * 2
    for shift in (2, -2, m - 2, 2 - m):
        assert call(lib, "ssd_linear", linear_prm(), res=FAKE, out=FAKE + shift, ws_bytes=0) == BADARG
    assert call(lib, "ssd_linear", linear_prm(residual_stride=97), res=FAKE, out=FAKE, ws_bytes=0) == BADARG
    for stride in (0, 96):
        assert call(lib, "ssd_linear", linear_prm(residual_stride=stride), res=FAKE, out=FAKE, ws_bytes=0) == WS_SMALL
    b = dict(dsum=FAKE, ws_bytes=0)
    assert call(lib, "ssd_rms_norm_backward", norm_prm(), dres=FAKE + 2, **b) == BADARG
    assert call(lib, "ssd_rms_norm_backward", norm_prm(), dres=FAKE, **b) == WS_SMALL
    s = 2 * 64 * 4
    for shift in (0, 4, s - 4, 4 - s):
        assert call(lib, "ssd_gated_recurrence", rec_prm(), h0=FAKE, fin=FAKE + shift, ws_bytes=0) == BADARG
        assert call(lib, "ssd_gated_recurrence_backward", rec_prm(), dfin=FAKE, dh0=FAKE + shift, ws_bytes=0) == BADARG
    assert call(lib, "ssd_gated_recurrence", rec_prm(), h0=FAKE, fin=FAKE + s, ws_bytes=0) == WS_SMALL


@pytest.mark.parametrize("name,size,prm", [
    ("ssd_rms_norm_backward", "ssd_rms_norm_backward_workspace_size", norm_prm(rows=5000)),
    ("ssd_linear", "ssd_linear_workspace_size", linear_prm()),
    ("ssd_linear", "ssd_linear_workspace_size", linear_prm(width=2049, x_stride=3001)),
    ("ssd_linear_backward", "ssd_linear_backward_workspace_size", linear_prm(width=77, outs=33)),
    ("ssd_gated_recurrence", "ssd_gated_recurrence_workspace_size", rec_prm(seqlen=5000)),
    ("ssd_gated_recurrence_backward", "ssd_gated_recurrence_backward_workspace_size", rec_prm(seqlen=5000))])
def test_workspaces(lib, name, size, prm):
    n = getattr(lib, size)(ctypes.byref(prm))
    assert n > 0 and n % 256 == 0
    assert call(lib, name, prm, ws_bytes=n - 1) == WS_SMALL
    prm.struct_size = 0
    assert getattr(lib, size)(ctypes.byref(prm)) == 0


def test_saved_states(lib):
    size = lib.ssd_gated_recurrence_saved_size
    for L, tiles in ((1, 1), (64, 1), (65, 2), (1000, 16)):
        assert size(ctypes.byref(rec_prm(seqlen=L))) == 2 * tiles * 64 * 4


def test_struct_layouts(tmp_path):
    """Every field at the header's offset, as gcc lays it out."""
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    structs = {"ssd_norm_params_t": ssd.NormParams, "ssd_linear_params_t": ssd.LinearParams,
               "ssd_recurrence_params_t": ssd.RecurrenceParams}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "mamba_ssd.h"', "int main(void) {"]
    for c, py in structs.items():
        lines.append('printf("%%zu\\n", sizeof(%s));' % c)
        lines += ['printf("%%zu\\n", offsetof(%s, %s));' % (c, f) for f, _ in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, stdout=subprocess.PIPE).stdout.split()]
    want = []
    for py in structs.values():
        want.append(ctypes.sizeof(py))
        want += [getattr(py, f).offset for f, _ in py._fields_]
    assert got == want


def test_the_binding_refuses_what_it_cannot_pass():
    x, w = torch.zeros(2, 8), torch.zeros(8)
    for f in (lambda: ssd.rms_norm(x, w), lambda: ssd.linear(x, torch.zeros(3, 8)),
              lambda: ssd.gated_recurrence(x[:, None], x[:, None], w), lambda: ssd.linear_backward(x, x, torch.zeros(8, 8)),
              lambda: ssd.rms_norm_backward(x, x, w), lambda: ssd.gated_recurrence_step(x, x, w, state=x)):
        with pytest.raises(ValueError, match="device tensors"):
            f()
    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        ssd.rms_norm(x.double(), w)
    with pytest.raises(ValueError, match="residual must be"):
        ssd.rms_norm(x.half(), w, x.bfloat16())
    with pytest.raises(ValueError, match="format"):
        ssd.rms_norm(x, w, format="int4")
    with pytest.raises(ValueError, match="out_dtype"):
        ssd.linear(x.to(torch.int8), torch.zeros(3, 8, dtype=torch.int8))
    with pytest.raises(ValueError, match="linear_backward takes"):
        ssd.linear_backward(x, x.to(torch.int8), torch.zeros(8, 8, dtype=torch.int8))
    with pytest.raises(ValueError, match="states must be"):
        ssd.gated_recurrence_step(x, x, w, state=x.to(torch.int32))
    with pytest.raises(ValueError, match=r"state must be \[nslots"):
        ssd.gated_recurrence_step(x, x, w, state=w)
    with pytest.raises(ValueError, match="nseq goes with seq_idx"):
        ssd.gated_recurrence(x[:, None], x[:, None], w, nseq=2)


def test_more_refusals_of_the_binding(monkeypatch):
    """Checks behind the one for device tensors, on tensors without a device's data."""
    monkeypatch.setattr(layer._s, "_on_gpu", lambda t, what: t.device)
    x, w, W = torch.zeros(2, 8), torch.zeros(8), torch.zeros(3, 8)
    cases = [(lambda: ssd.rms_norm(x[0], w), "at least 2 dimensions"), (lambda: ssd.rms_norm(x, w[:4]), "weight has shape"),
             (lambda: ssd.rms_norm(x, w.half()), "weight must be torch.float32"),
             (lambda: ssd.rms_norm(x.t(), torch.zeros(2)), "elements of a row"),
             (lambda: ssd.rms_norm(x, w, torch.zeros(3, 8)), "residual has shape"),
             (lambda: ssd.rms_norm(x, w, residual_out=x), "goes with residual"),
             (lambda: ssd.rms_norm_backward(x.half(), x.bfloat16(), w), "s must be"),
             (lambda: ssd.linear(x, W.half()), "weight must be"), (lambda: ssd.linear(x, W[:, :4]), "weight has shape"),
             (lambda: ssd.linear(x, W[0]), r"\[outs, width\]"), (lambda: ssd.linear(x, W, activation="relu"), "activation"),
             (lambda: ssd.linear(x, W, residual=torch.zeros(2, 4)), "residual has shape"),
             (lambda: ssd.linear(x, W, torch.zeros(4)), "bias has shape"),
             (lambda: ssd.linear(x.to(torch.int32), W), "x must be"),
             (lambda: ssd.linear(x, W, out_dtype=torch.float64), "states must be"),
             (lambda: ssd.linear_backward(torch.zeros(2, 3), x, W, activation="silu"), "pre goes with"),
             (lambda: ssd.linear_backward(torch.zeros(2, 4), x, W), "dout has shape"),
             (lambda: ssd.gated_recurrence(x[:, None], x[:, None], w, None, None, w), "in_bias goes with"),
             (lambda: ssd.gated_recurrence(x[:, None], x[:, None].half(), w), "gate must be"),
             (lambda: ssd.gated_recurrence(x, x, w), "x must have 3"),
             (lambda: ssd.gated_recurrence(x[:, None], x[:, None], w, seq_idx=torch.zeros(2, 1)), "nseq >= 1"),
             (lambda: ssd.gated_recurrence(x[:, None], x[:, None], w, initial_state=torch.zeros(1, 8)), "initial_state has shape")]
    for f, match in cases:
        with pytest.raises(ValueError, match=match):
            f()


def test_refused_parameters_keep_their_status(monkeypatch):
    monkeypatch.setattr(layer._s, "_on_gpu", lambda t, what: t.device)
    with pytest.raises(ssd.SSDError) as e:
        ssd.linear(torch.zeros(0, 8), torch.zeros(3, 8))
    assert e.value.code == SHAPE
    with pytest.raises(ssd.SSDError) as e:
        ssd.rms_norm_backward(torch.zeros(2, 20000), torch.zeros(2, 20000), torch.zeros(20000))
    assert e.value.code == UNSUP


def test_counts_that_the_parameter_blocks_cannot_hold(monkeypatch):
    """Sizes from 2^31 are refused, not cut to 32 bits (tensors without data, so that they take no memory)."""
    monkeypatch.setattr(layer._s, "_on_gpu", lambda t, what: t.device)
    n = 2**31 + 5
    new = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="meta")  # noqa: E731
    w = new(8)
    cases = [(lambda: ssd.rms_norm(new(1, n), new(n)), "width"), (lambda: ssd.linear(new(n, 8), new(3, 8)), "rows"),
             (lambda: ssd.linear(new(2, n), new(3, n)), "width"), (lambda: ssd.linear(new(2, 8), new(n, 8)), "outs"),
             (lambda: ssd.linear_backward(new(n, 3), new(n, 8), new(3, 8)), "rows"),
             (lambda: ssd.gated_recurrence(new(n, 1, 8), new(n, 1, 8), w), "batch"),
             (lambda: ssd.gated_recurrence(new(1, n, 8), new(1, n, 8), w), "seqlen"),
             (lambda: ssd.gated_recurrence(new(1, 1, n), new(1, 1, n), new(n)), "channels"),
             (lambda: ssd.gated_recurrence(new(1, 1, 8), new(1, 1, 8), w, seq_idx=new(1, 1, dtype=torch.int32), nseq=n), "nseq"),
             (lambda: ssd.gated_recurrence_step(new(n, 8), new(n, 8), w, state=new(4, 8)), "batch"),
             (lambda: ssd.gated_recurrence_step(new(2, 8), new(2, 8), w, state=new(n, 8)), "nseq")]
    for f, name in cases:
        with pytest.raises(ValueError, match=name + " must be below"):
            f()
