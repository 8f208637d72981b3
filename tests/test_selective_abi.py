"""Refusals of the causal convolution, the selective scan and the 8-bit state cache, without a GPU: every C call
here fails exactly one host check (fake aligned addresses), so nothing is launched; and the binding's
structs have the header's layout."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import mamba_ssd_prefill_amd as ssd
from mamba_ssd_prefill_amd import selective

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULLP, SHAPE, UNSUP, MISAL, WS_SMALL, HIP, TIMEOUT, BADARG = range(9)
FAKE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return ssd.load_library()


def conv_prm(**kw):
    p = dict(batch=2, seqlen=30, channels=64, width=4, in_dtype=2, silu=1, nseq=0, split_a=64, split_b=64, x_stride=0)
    p.update(kw)
    return ssd.ConvParams(ctypes.sizeof(ssd.ConvParams), *p.values())


def scan_prm(**kw):
    p = dict(batch=2, seqlen=30, channels=64, dstate=16, ngroups=1, in_dtype=2, state_dtype=0, dt_softplus=1, nseq=0,
             x_stride=0, dt_stride=0, z_stride=0, B_stride=0, C_stride=0)
    p.update(kw)
    return ssd.ScanParams(ctypes.sizeof(ssd.ScanParams), *p.values())


def cache_prm(**kw):
    p = dict(batch=2, nslots=4, elems=1024, group=64, format=0, state_dtype=0)
    p.update(kw)
    return ssd.CacheParams(ctypes.sizeof(ssd.CacheParams), *p.values())


# the pointer arguments of each entry point, and those that may be NULL in the calls below
ARGS = {
    "ssd_causal_conv": ("x w bias seq h0 out0 out1 out2 fin", "bias seq h0 out1 out2 fin"),
    "ssd_causal_conv_backward": ("dout0 dout1 dout2 dfin x w bias seq h0 dx dw db dh0 ws", "dout1 dout2 dfin bias seq h0 db dh0"),
    "ssd_causal_conv_step": ("x w bias state slots out0 out1 out2", "bias slots out1 out2"),
    "ssd_selective_scan": ("x dt A B C D bias z seq h0 out fin saved ws", "D bias z seq h0 fin saved"),
    "ssd_selective_scan_backward": ("dout dfin x dt A B C D bias z seq h0 saved dx ddt dA dB dC dD db dz dh0 ws",
                                    "dfin D bias z seq h0 dD db dz dh0"),
    "ssd_selective_scan_step": ("x dt A B C D bias z state slots out", "D bias z slots"),
    "ssd_state_cache_write": ("state slots codes scales", "slots"),
    "ssd_state_cache_read": ("codes scales slots state", "slots"),
}
PRM = {"ssd_causal": conv_prm, "ssd_select": scan_prm, "ssd_state_": cache_prm}


def params_for(name, **kw):
    if name.endswith("_step"):
        kw = dict(dict(seqlen=1, nseq=2), **kw)
    return PRM[name[:10]](**kw)


def call(lib, name, prm, ws_bytes=1 << 40, **over):
    fields = ARGS[name][0].split()
    vals = {f: FAKE * (i + 1) for i, f in enumerate(fields)}
    vals["seq"] = None
    vals["slots"] = None
    vals.update(over)
    a = [vals[f] for f in fields]
    if "ws" in fields:
        a.append(ws_bytes)
    return getattr(lib, name)(ctypes.byref(prm) if prm is not None else None, *a, None)


@pytest.mark.parametrize("name", sorted(ARGS))
def test_null_pointers(lib, name):
    assert call(lib, name, None) == NULLP
    fields, free = (s.split() for s in ARGS[name])
    for f in fields:
        if f not in free:
            assert call(lib, name, params_for(name), **{f: None}) == NULLP, f
    if name == "ssd_selective_scan_backward":
        assert call(lib, name, params_for(name), dz=None) == NULLP
        assert call(lib, name, params_for(name), z=None) == BADARG


ALIGN = {"h0": 16, "fin": 16, "dfin": 16, "dh0": 16, "saved": 16, "state": 16, "codes": 16, "A": 16, "ws": 256, "B": 4, "C": 4,
         "dB": 16, "dC": 16}


@pytest.mark.parametrize("name", sorted(ARGS))
def test_misaligned(lib, name):
    for i, f in enumerate(ARGS[name][0].split()):
        conv = "conv" in name
        a = 2 if conv and f in ("h0", "fin", "dfin", "dh0", "state") else ALIGN.get(f, 4 if f in (
            "w", "bias", "seq", "D", "dw", "db", "dD", "dA", "slots", "scales") else 2)
        if f in ("out1", "out2", "dout1", "dout2"):
            continue
        kw = dict(nseq=2) if f in ("seq", "slots") and "cache" not in name else {}
        assert call(lib, name, params_for(name, **kw), **{f: FAKE * (i + 1) + a // 2}) == MISAL, (f, a)
    if "conv" in name:  # a range with channels needs its tensor, aligned
        prm = params_for(name, split_a=10, split_b=20)
        pre = "dout" if "backward" in name else "out"
        for k in (1, 2):
            assert call(lib, name, prm, **{pre + str(k): None}) == NULLP
            assert call(lib, name, prm, **{pre + str(k): FAKE + 1}) == MISAL


@pytest.mark.parametrize("name", ["ssd_causal_conv", "ssd_causal_conv_backward", "ssd_causal_conv_step"])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), SHAPE), (dict(channels=0), SHAPE), (dict(seqlen=0), SHAPE), (dict(width=1), UNSUP),
    (dict(width=5), UNSUP), (dict(in_dtype=3), BADARG), (dict(silu=2), BADARG), (dict(split_a=65), SHAPE),
    (dict(split_a=-1), SHAPE), (dict(split_a=20, split_b=10), SHAPE), (dict(split_b=65), SHAPE), (dict(x_stride=63), SHAPE),
    (dict(x_stride=-64), SHAPE), (dict(batch=1 << 20, seqlen=1 << 12), SHAPE)])
def test_conv_parameters(lib, name, kw, code):
    if name.endswith("_step") and "seqlen" in kw and kw["seqlen"] != 0:
        kw = dict(seqlen=2)
    assert call(lib, name, params_for(name, **kw)) == code


@pytest.mark.parametrize("name", ["ssd_selective_scan", "ssd_selective_scan_backward", "ssd_selective_scan_step"])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), SHAPE), (dict(channels=0), SHAPE), (dict(seqlen=0), SHAPE), (dict(ngroups=0), SHAPE),
    (dict(ngroups=3), SHAPE), (dict(dstate=0), SHAPE), (dict(dstate=4), UNSUP), (dict(dstate=24), UNSUP),
    (dict(dstate=128), UNSUP), (dict(in_dtype=-1), BADARG), (dict(state_dtype=3), BADARG), (dict(dt_softplus=2), BADARG),
    (dict(x_stride=10), SHAPE), (dict(dt_stride=-1), SHAPE), (dict(z_stride=63), SHAPE), (dict(B_stride=15), SHAPE),
    (dict(C_stride=17), MISAL), (dict(B_stride=19), MISAL), (dict(batch=1 << 20, seqlen=1 << 12), SHAPE),
    (dict(channels=1 << 28), SHAPE)])
def test_scan_parameters(lib, name, kw, code):
    if name.endswith("_step") and "seqlen" in kw and kw["seqlen"] != 0:
        kw = dict(seqlen=2)
    assert call(lib, name, params_for(name, **kw)) == code


@pytest.mark.parametrize("name", ["ssd_state_cache_write", "ssd_state_cache_read"])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), SHAPE), (dict(nslots=0), SHAPE), (dict(elems=0), SHAPE), (dict(elems=1000), SHAPE), (dict(group=0), SHAPE),
    (dict(group=48), UNSUP), (dict(group=256), UNSUP), (dict(format=2), BADARG), (dict(state_dtype=9), BADARG),
    (dict(batch=5), SHAPE), (dict(elems=1 << 40), SHAPE)])
def test_cache_parameters(lib, name, kw, code):
    assert call(lib, name, cache_prm(**kw)) == code


@pytest.mark.parametrize("name", sorted(ARGS))
def test_short_struct(lib, name):
    p = params_for(name)
    p.struct_size -= 1
    assert call(lib, name, p) == BADARG


def test_packed_input_and_pools_need_their_number_of_states(lib):
    for name in ("ssd_causal_conv", "ssd_causal_conv_backward", "ssd_selective_scan", "ssd_selective_scan_backward"):
        assert call(lib, name, params_for(name, nseq=0), seq=FAKE) == SHAPE
    for name in ("ssd_causal_conv_step", "ssd_selective_scan_step"):
        assert call(lib, name, params_for(name, nseq=0), slots=FAKE) == SHAPE
        assert call(lib, name, params_for(name, nseq=3)) == SHAPE  # without slots: one state per row


def test_states_in_place_are_refused_for_prompts(lib):
    for name in ("ssd_causal_conv", "ssd_selective_scan"):
        assert call(lib, name, params_for(name), h0=FAKE, fin=FAKE) == BADARG


def test_workspaces(lib):
    for name, size in (("ssd_causal_conv_backward", lib.ssd_causal_conv_backward_workspace_size),
                       ("ssd_selective_scan", lib.ssd_selective_scan_workspace_size),
                       ("ssd_selective_scan_backward", lib.ssd_selective_scan_backward_workspace_size)):
        p = params_for(name)
        n = size(ctypes.byref(p))
        assert n > 0 and n % 256 == 0
        assert call(lib, name, p, ws_bytes=n - 1) == WS_SMALL
        assert size(ctypes.byref(params_for(name, batch=0))) == 0 and size(None) == 0
    assert lib.ssd_selective_scan_saved_size(ctypes.byref(scan_prm(seqlen=33))) == 2 * 5 * 64 * 16 * 4
    assert lib.ssd_selective_scan_saved_size(ctypes.byref(scan_prm(seqlen=33, dstate=64))) == 2 * 5 * 64 * 64 * 4
    assert lib.ssd_selective_scan_saved_size(ctypes.byref(scan_prm(dstate=24))) == 0


def test_struct_layouts(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    pairs = [("ssd_conv_params_t", ssd.ConvParams), ("ssd_scan_params_t", ssd.ScanParams), ("ssd_cache_params_t", ssd.CacheParams)]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "mamba_ssd.h"\nint main(void) {\n'
    for c, cls in pairs:
        src += '    printf("%%zu\\n", sizeof(%s));\n' % c
        for f, _ in cls._fields_:
            src += '    printf("%%zu\\n", offsetof(%s, %s));\n' % (c, f)
    (tmp_path / "s.c").write_text(src + "    return 0;\n}\n")
    subprocess.run([gcc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(tmp_path / "s.c"), "-o", str(tmp_path / "s")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True).stdout.split()]
    want = []
    for _, cls in pairs:
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def test_the_binding_refuses_what_it_cannot_pass():
    z = torch.zeros
    with pytest.raises(ValueError, match="device"):
        ssd.causal_conv(z(1, 4, 8), z(8, 4))
    with pytest.raises(ValueError, match="device"):
        ssd.selective_scan(z(1, 4, 8), z(1, 4, 8), z(8, 8), z(1, 4, 1, 8), z(1, 4, 1, 8))
    with pytest.raises(ValueError, match="device"):
        ssd.state_cache_write(z(1, 64), *ssd.state_cache(1, (64,), device="cpu"))
    with pytest.raises(ValueError, match="nseq"):
        ssd.causal_conv(z(1, 4, 8), z(8, 4), seq_idx=z(1, 4, dtype=torch.int32))
    with pytest.raises(ValueError, match="nseq"):
        ssd.selective_scan(z(1, 4, 8), z(1, 4, 8), z(8, 8), z(1, 4, 1, 8), z(1, 4, 1, 8), nseq=3)
    with pytest.raises(ValueError, match="group"):
        ssd.state_cache(2, (40,), device="cpu")
    with pytest.raises(ValueError, match="format"):
        ssd.state_cache(2, (64,), format="int4", device="cpu")
    with pytest.raises(ValueError, match="float"):
        ssd.selective_scan(z(1, 4, 8), z(1, 4, 8), z(8, 8), z(1, 4, 1, 8), z(1, 4, 1, 8), state_dtype=torch.float64)


def test_row_views():
    """The distance between rows that the binding finds in views, and the views it refuses."""
    rows = lambda t, lead=2: selective._rows("x", t, t.device, t.dtype, t.shape, lead)  # noqa: E731
    u = torch.zeros(3, 5, 20)
    assert rows(u) == 0 and rows(u[..., 4:12]) == 20 and rows(u[:1, 1:4, :8]) == 20 and rows(u[:, :1, :8]) == 100
    assert rows(u[:1, :1, :8]) == 0 and rows(u[:, 2], 1) == 100
    assert rows(u[..., :12].unflatten(-1, (3, 4))) == 20
    for bad in (u[:, :, ::2], u[:, 1:4, :8], u.transpose(1, 2), u[..., :1].expand(3, 5, 4), u[:, ::2, :8],
                torch.zeros(1, 1, 8).expand(3, 5, 8)):
        with pytest.raises(ValueError):
            rows(bad)


def test_refused_parameters_keep_their_status():
    """A plan that the library refuses raises with the library's own status (CPU: the checks come before any call)."""
    prm = scan_prm(seqlen=0)
    with pytest.raises(ssd.SSDError) as e:
        selective._Plan("ssd_selective_scan", prm, torch.device("cpu"), spaces=("ssd_selective_scan_workspace_size",))
    assert e.value.code == SHAPE
    with pytest.raises(ssd.SSDError) as e:
        selective._Plan("ssd_selective_scan", scan_prm(dstate=24), torch.device("cpu"),
                        spaces=("ssd_selective_scan_workspace_size",))
    assert e.value.code == UNSUP


def test_meta_tells_calls_apart():
    """Equal keys for tensors that pass the same checks, others for another size, stride, type or place; addresses as
    they are; other things than tensors are refused."""
    from mamba_ssd_prefill_amd._meta import meta
    x, y = torch.zeros(2, 3), torch.ones(2, 3)
    key, (px, none, pv) = meta(x, None, x[:, 1:])
    assert (px, none, pv) == (x.data_ptr(), None, x.data_ptr() + 4)
    assert key == meta(y, None, y[:, 1:])[0]
    keys = [meta(*a)[0] for a in ((x,), (x.t(),), (x.half(),), (x.view(6),), (x, None), (None, x), (None, None), (),
                                  (x[:, :2],), (x[:1],), (x.view(1, 2, 3),))]
    assert len(set(keys)) == len(keys)
    for bad in (3, "x", [x]):
        with pytest.raises(TypeError):
            meta(x, bad)
    with pytest.raises(ValueError):
        meta(x.to_sparse())


def test_new_tensors_of_layouts():
    from mamba_ssd_prefill_amd._meta import meta, new
    lay = selective._layout((2, 3, 5), torch.bfloat16, torch.device("cpu"))
    a, b = new(lay, meta(torch.zeros(4, 6)[:, :3])[0])
    assert a.shape == (2, 3, 5) and a.dtype == torch.bfloat16 and a.is_contiguous()
    assert b.shape == (4, 3) and b.stride() == (6, 1) and b.dtype == torch.float32
    assert lay == meta(a)[0] and new() == ()
    for bad in (b"", lay[:-8], lay + b"x" * 8, "x", meta(a, a)[0], meta(None)[0]):
        with pytest.raises(ValueError):
            new(bad)


@pytest.mark.parametrize("name,fits,over", [
    # (a missing tensor is found after the sizes)
    ("ssd_causal_conv", dict(batch=1, seqlen=(1 << 31) - 256), dict(batch=1, seqlen=(1 << 31) - 1)),
    ("ssd_causal_conv", dict(batch=1 << 12, seqlen=1 << 16, channels=448, split_a=448, split_b=448),
     dict(batch=1 << 12, seqlen=1 << 16, channels=449, split_a=449, split_b=449)),
    ("ssd_causal_conv_backward", dict(batch=1, seqlen=(1 << 31) - 256, channels=1, split_a=1, split_b=1),
     dict(batch=1 << 26, seqlen=1, channels=1, split_a=1, split_b=1)),
    ("ssd_causal_conv_step", dict(batch=(1 << 26) - 4, nseq=(1 << 26) - 4), dict(batch=1 << 26, nseq=1 << 26)),
    ("ssd_selective_scan", dict(batch=(1 << 23) - 1, seqlen=200), dict(batch=1 << 23, seqlen=200)),
    ("ssd_selective_scan_backward", dict(batch=1 << 20, seqlen=120), dict(batch=1 << 20, seqlen=128)),
    ("ssd_selective_scan_backward", dict(seqlen=1 << 20, dstate=64, ngroups=8), dict(seqlen=1 << 20, dstate=64, ngroups=16)),
    ("ssd_selective_scan_step", dict(batch=(1 << 22) - 1, nseq=(1 << 22) - 1, dstate=64),
     dict(batch=1 << 22, nseq=1 << 22, dstate=64)),
    ("ssd_state_cache_write", dict(batch=1 << 13, nslots=1 << 13, elems=2047 * 2048), dict(batch=1 << 13, nslots=1 << 13, elems=2047 * 2048 + 2048)),
    ("ssd_state_cache_read", dict(elems=(1 << 34) - 4096), dict(elems=1 << 34)),
])
def test_a_launch_s_lanes_are_bounded(lib, name, fits, over):
    first = ARGS[name][0].split()[0]
    assert call(lib, name, params_for(name, **fits), **{first: None}) == NULLP
    assert call(lib, name, params_for(name, **over), **{first: None}) == SHAPE


def test_library_calls_by_address():
    from mamba_ssd_prefill_amd._meta import call
    for n in (0, 1, 5, 6, 7, 17, 26, 32):
        seen = []
        f = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_size_t] * n)(lambda *a: seen.append(a) or -n)
        where = ctypes.cast(f, ctypes.c_void_p).value
        args = [(1 << 63) + 7 * i if i % 3 else None for i in range(n)]
        assert call(where, *args) == -n
        assert seen == [tuple(a or 0 for a in args)]
    for bad in ((), (where,) + (0,) * 33):
        with pytest.raises(TypeError):
            call(*bad)
    with pytest.raises(ValueError):
        call(0, 1)
    for bad in ("x", -1, 1 << 64, 1.5):
        with pytest.raises((TypeError, OverflowError)):
            call(where, bad)


@pytest.mark.parametrize("over", [0, 1, 47, 55, 62])
def test_scan_tiles_of_the_longest_rows_stay_in_range(lib, over):
    """A row's tiles and the tokens a tile reaches behind it are 32-bit numbers: the last 63 lengths are refused (the
    backward's sums stop earlier)."""
    one = dict(batch=1, channels=1, dstate=8)
    assert call(lib, "ssd_selective_scan", scan_prm(seqlen=(1 << 31) - 64, **one), x=None) == NULLP
    assert call(lib, "ssd_selective_scan", scan_prm(seqlen=(1 << 31) - 1 - over, **one), x=None) == SHAPE
    assert lib.ssd_selective_scan_saved_size(ctypes.byref(scan_prm(seqlen=(1 << 31) - 64, **one))) == ((1 << 28) - 8) * 8 * 4
    for size in (lib.ssd_selective_scan_saved_size, lib.ssd_selective_scan_workspace_size,
                 lib.ssd_selective_scan_backward_workspace_size):
        assert size(ctypes.byref(scan_prm(seqlen=(1 << 31) - 1 - over, **one))) == 0


@pytest.mark.parametrize("width,most", [(2, (1 << 30) // 3), (3, (1 << 30) // 4 - 1), (4, (1 << 30) // 5)])
def test_lanes_of_the_convolution_backward_s_sums_are_bounded(lib, width, most):
    """k_conv_sums takes four lanes a value of dw and dbias: (width + 1) * channels of them stay below 2^30."""
    name = "ssd_causal_conv_backward"
    at = lambda n: conv_prm(batch=1, seqlen=1, channels=n, split_a=n, split_b=n, width=width)  # noqa: E731
    most = most // 64 * 64
    assert call(lib, name, at(most), x=None) == NULLP
    assert call(lib, name, at(most + 64), x=None) == SHAPE
    assert lib.ssd_causal_conv_backward_workspace_size(ctypes.byref(at(most))) > 0
    assert lib.ssd_causal_conv_backward_workspace_size(ctypes.byref(at(most + 64))) == 0
    assert call(lib, "ssd_causal_conv", at(most + 64), x=None) == NULLP


@pytest.mark.parametrize("field", ["x_stride", "dt_stride", "z_stride", "B_stride", "C_stride"])
def test_rows_of_a_step_may_lie_far_apart(lib, field):
    """One token of every row of a long joint projection (x = u[:, t, :D]): rows 2^24 elements and more apart, which the
    prompt's tiles do not reach."""
    name = "ssd_selective_scan_step"
    for far in (1 << 24, 200000 * 10240, (1 << 31) - 2):
        assert call(lib, name, params_for(name, **{field: far}), x=None) == NULLP
    assert call(lib, name, params_for(name, **{field: 1 << 31}), x=None) == SHAPE
    if field[0] in "BC":
        assert call(lib, name, params_for(name, **{field: (1 << 24) + 1}), x=None) == MISAL
    for name in ("ssd_selective_scan", "ssd_selective_scan_backward"):
        assert call(lib, name, params_for(name, **{field: 1 << 24}), **{ARGS[name][0].split()[0]: None}) == SHAPE


@pytest.fixture
def plans(monkeypatch):
    """The binding's store of plans, empty, and as it was afterwards."""
    for name in ("_PLANS", "_BEFORE"):
        monkeypatch.setattr(selective, name, {}, raising=False)
    return lambda key: selective._PLANS.get(key) or selective._older(key)


def test_plans_in_use_outlive_new_sizes(plans):
    """A server's step keeps its plan while prompts of thousands of lengths come by."""
    step = object()
    selective._keep(("scan step", b"sizes", True), step)
    for i in range(5 * selective._MAX_PLANS):
        selective._keep(("scan", b"%d" % i, None), object())
        if i % 7 == 0:
            assert plans(("scan step", b"sizes", True)) is step, i
    assert len(selective._PLANS) + len(selective._BEFORE) <= selective._MAX_PLANS
    assert plans(("scan", b"0", None)) is None


def test_plans_are_kept_under_values_alone(plans):
    """An argument that is told apart by its identity (a tensor as a flag or a count) is never looked up again: its value
    may be another by then."""
    import numpy as np
    plan = object()
    for kept in (("conv", b"", "silu", 3, (4, 5)), ("scan", b"", True, None, torch.float16), ("scan", b"", np.int64(1), None)):
        assert selective._keep(kept, plan) is plan and plans(kept) is plan
    for flag in (torch.tensor(True), (2, torch.tensor(3)), [1]):
        key = ("scan", b"", flag, None, None)
        assert selective._keep(key, plan) is plan
        assert not any(k[2] is flag for k in [*selective._PLANS, *selective._BEFORE])


def test_library_calls_raise_the_versions_of_written_tensors():
    """A tensor among a call's arguments stands for its address and is taken to be written: its version goes up, as with
    torch's own writes in place (a view's base's too; tensors of the inference mode have none)."""
    from mamba_ssd_prefill_amd._meta import call
    seen = []
    f = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_size_t] * 4)(lambda *a: seen.append(a) or 0)
    where = ctypes.cast(f, ctypes.c_void_p).value
    base = torch.zeros(4, 6)
    with torch.inference_mode():
        inf = torch.zeros(3)
    other = torch.zeros(2)
    assert call(where, base[1:], other.data_ptr(), None, inf) == 0
    assert seen == [(base.data_ptr() + 24, other.data_ptr(), 0, inf.data_ptr())]
    assert base._version == 1 and other._version == 0
    with pytest.raises(TypeError):
        call(base, 1)
    with pytest.raises((RuntimeError, ValueError, NotImplementedError)):
        call(where, base.to_sparse(), 0, 0, 0)


def test_states_that_overlap_are_refused_for_prompts(lib):
    """A final state that lies partly over the initial one (shifted views of one pool): other workgroups still read that."""
    for name, size in (("ssd_causal_conv", 64 * 3 * 2), ("ssd_selective_scan", 64 * 16 * 4)):
        for S, kw, seq in ((2, {}, None), (5, dict(nseq=5), FAKE * 64)):
            prm = params_for(name, **kw)
            for d in (16, size, S * size - 16):
                for h0, fin in ((FAKE, FAKE + d), (FAKE + d, FAKE)):
                    assert call(lib, name, prm, seq=seq, h0=h0, fin=fin) == BADARG, (name, S, d)
        n = S * size  # next to each other: on to the next check
        if name == "ssd_selective_scan":
            assert call(lib, name, prm, seq=seq, h0=FAKE, fin=FAKE + n, ws_bytes=0) == WS_SMALL
            assert call(lib, name, prm, seq=seq, h0=FAKE + n, fin=FAKE, ws_bytes=0) == WS_SMALL
