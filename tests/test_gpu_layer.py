"""GPU tests of the residual norm, the matrix product with its epilogue and the gated recurrence against the 64-bit
references of layer_ref.py.  Tolerances are the bounds derived there: half a step of the output's type plus K u S, K the
most roundings on a path from an input to the output, S the sum of absolute products:
  norm: a lane adds at most 64 squares, 6 exchanges and 16 waves follow, half of it for the root, 14 for the root itself, the
        division, the products and the addition: 60 relative to the output.  Gradients: two such sums, 200; dw: one more a row
  product: a matrix instruction's additions are within two roundings each: 2 a product, 20 for scales, bias, residual; 60 for an
        activation (whose slope is below 1.2).  Gradients: the same, and half a step of the type for dpre behind an activation
  recurrence: a gate is right to 14 u at |v| below 8, which a decay's exponent takes times |A|: 14 + 14 |A| a token, 100 for
        the addition; gradients twice that and 200, sums one more a token
"""
import pytest
import torch

import layer_ref as ref
import mamba_ssd_prefill_amd as ssd
from gpu_common import require_gpu, say
from test_gpu_selective import cuda, gen, packing, strided

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def dev():
    return require_gpu()


def rn(g, *shape):
    return torch.randn(*shape, generator=g)


# ---- residual norm --------------------------------------------------------------------------------
NORM = [
    # (rows, D, dtype, residual, format, strided)
    (1, 1, "f32", None, None, False),
    (3, 7, "bf16", "same", None, True),
    (5, 64, "f16", "f32", "int8", False),
    (1, 2560, "bf16", "same", None, False),
    (1030, 511, "f16", "same", "e4m3", True),
    (1030, 512, "bf16", "f32", None, True),
    (1025, 513, "f32", "same", "int8", False),
    (6, 1111, "f16", None, "e4m3", True),
    (1029, 1300, "f32", None, None, False),
    (1027, 2563, "bf16", "same", "int8", False),
    (4, 4100, "f32", "same", "e4m3", False),
    (3, 8193, "bf16", "f32", "e4m3", True),
    (2, 16384, "f16", "same", "int8", False),
    (2, 16384, "f32", "same", None, False),
    (2, 16383, "bf16", None, None, True),
]


def norm_case(case, seed):
    M, D, dtype, res, fmt, stride = case
    g, t = gen(seed), DT[dtype]
    x = rn(g, M, D).to(t)
    r = None if res is None else (3 * rn(g, M, D)).to(t if res == "same" else torch.float32)
    w = 1 + 0.2 * rn(g, D)
    view = (lambda v: strided(v[:, None].cuda()).squeeze(1)) if stride else cuda  # noqa: E731
    return x, r, w, view(x), None if r is None else view(r), w.cuda()


def check_codes(codes, scales, y, fmt):
    scales, most = scales.cpu().double(), 127 if fmt == "int8" else 448
    want = y.abs().amax(-1) / most
    assert ((scales - want).abs() <= 61 * ref.U * want).all()
    q = y / scales[..., None]
    held = codes.float().cpu().double()
    tol = ref.code_step(q, fmt) / 2 + 62 * ref.U * q.abs()
    assert ((held - q).abs() <= tol).all()


@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm(case):
    say("norm", case)
    M, D, dtype, res, fmt, _ = case
    x, r, w, xg, rg, wg = norm_case(case, 31)
    got = ssd.rms_norm(xg, wg, rg, eps=1e-5, format=fmt)
    torch.cuda.synchronize()
    got = got if isinstance(got, tuple) else (got,)
    s, y = ref.norm(x, r, w, 1e-5)
    if fmt is None:
        ref.close(got[0], y, y.abs(), 60, x.dtype, "norm")
    else:
        assert got[0].dtype == (torch.int8 if fmt == "int8" else torch.float8_e4m3fn) and got[0].shape == x.shape
        check_codes(got[0], got[1], y, fmt)
    if res is not None:
        ref.close(got[-1], s, s.abs(), 1, r.dtype, "sum")
    assert len(got) == 1 + (fmt is not None) + (res is not None)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("M,D,dtype,res", [(1500, 2560, "bf16", "f32"), (1500, 2560, "f16", "same"), (4000, 1000, "bf16", "same"),
                                           (2500, 1111, "f32", "f32"), (400, 8191, "f16", None),
                                           (300, 12000, "f32", "same")], ids=str)
def test_norm_codes_next_to_borders(M, D, dtype, res, fmt):
    """Millions of values, of which some come within fp32's steps of a border of two codes: each takes the code of the 64-bit
    definition.  The sum with the residual is in fp32; behind it a value is right to the roundings of 64 bits, D of them and
    10: far below 2^-36.  The scale is right to half a step of fp32, and the quotient is by the scale as returned."""
    say("codes next to borders", M, D, dtype, res, fmt)
    g, t, eps = gen(34), DT[dtype], 2.0**-17
    x, w = rn(g, M, D).to(t), 1 + 0.2 * rn(g, D)
    r = None if res is None else (3 * rn(g, M, D)).to(t if res == "same" else torch.float32)
    codes, scales, *_ = ssd.rms_norm(x.cuda(), w.cuda(), cuda(r), eps=eps, format=fmt)
    torch.cuda.synchronize()
    _, y = ref.norm(x.float() if r is None else x.float() + r.float(), None, w, eps)
    want, scales = y.abs().amax(-1) / (127 if fmt == "int8" else 448), scales.cpu().double()
    assert ((scales - want).abs() <= (ref.U + 2.0**-36) * want).all()
    q = y / scales[..., None]
    off = (codes.float().cpu().double() - q).abs() - ref.code_step(q, fmt) / 2
    assert (off <= 2.0**-36 * q.abs()).all(), "%d codes" % int((off > 2.0**-36 * q.abs()).sum())


@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm_backward(case):
    say("norm backward", case)
    M, D, dtype, res, _, _ = case
    x, r, w, xg, rg, wg = norm_case(case, 32)
    g = gen(33)
    s = x if r is None else (x.double() + r.double()).to(r.dtype)
    sg = strided(s[:, None].cuda()).squeeze(1) if case[5] else s.cuda()
    dout, dsum = rn(g, M, D).to(x.dtype), None if r is None else rn(g, M, D).to(s.dtype)
    a, b = (ssd.rms_norm_backward(dout.cuda(), sg, wg, eps=1e-5, dresidual=cuda(dsum)) for _ in range(2))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))  # a fixed order of summation
    ds, dw = ref.norm_grads(dout, s, w, dsum, 1e-5)
    Sd, Sw = ref.norm_grads(dout, s, w, dsum, 1e-5, absolute=True)
    ref.close(a.dx, ds, Sd, 200, x.dtype, "dx")
    ref.close(a.dresidual, ds, Sd, 200, s.dtype, "dresidual")
    ref.close(a.dweight, dw, Sw, 70 + M, torch.float32, "dweight")
    assert (a.dx is a.dresidual) == (s.dtype == x.dtype)


def test_norm_of_more_rows_than_workgroups():
    M, D = 4 * (1 << 20) + 5, 2
    x = torch.randn(M, D, device="cuda").half()
    w = torch.tensor([1.5, -0.5], device="cuda")
    y = ssd.rms_norm(x, w)
    _, want = ref.norm(x, None, w, 1e-5)
    ref.close(y, want, want.abs(), 60, x.dtype, "norm")
    dout = torch.randn(M, D, device="cuda").half()
    got = ssd.rms_norm_backward(dout, x, w)
    ds, dw = ref.norm_grads(dout, x, w, None, 1e-5)
    Sd, Sw = ref.norm_grads(dout, x, w, None, 1e-5, absolute=True)
    ref.close(got.dx, ds, Sd, 200, x.dtype, "dx")
    ref.close(got.dweight, dw, Sw, 70 + M, torch.float32, "dweight")


@pytest.mark.parametrize("eps", [0.0, 1e-39, 2.0**-130])
@pytest.mark.parametrize("D", [64, 1500])
def test_norm_of_subnormal_squares(D, eps):
    """Rows of 2^-66 and the like (their squares are exact), and of zeros where eps alone stands under the root."""
    g = gen(6)
    sign = torch.where(rn(g, 4, D) > 0, 1.0, -1.0)
    x, w, dout = sign * 2.0 ** torch.tensor([[-66.0], [-62.0], [-70.0], [-64.0]]), rn(g, D), rn(g, 4, D)
    if eps:
        x[3] = 0
    eps = float(torch.tensor(eps))
    y = ssd.rms_norm(x.cuda(), w.cuda(), eps=eps)
    _, want = ref.norm(x, None, w, eps)
    ref.close(y, want, want.abs(), 60, torch.float32, "norm")
    got = ssd.rms_norm_backward(dout.cuda(), x.cuda(), w.cuda(), eps=eps)
    (ds, dw), (Sd, Sw) = (ref.norm_grads(dout, x, w, None, eps, absolute=k) for k in (False, True))
    ref.close(got.dx, ds, Sd, 200, torch.float32, "dx")
    ref.close(got.dweight, dw, Sw, 74, torch.float32, "dweight")


def test_norm_in_place_and_given_outputs():
    g = gen(5)
    x, r, w = rn(g, 2, 9, 300).bfloat16().cuda(), rn(g, 2, 9, 300).cuda(), rn(g, 300).cuda()
    y, s = ssd.rms_norm(x, w, r)
    out, held = torch.empty_like(x), r.clone()
    v = held._version
    y2, s2 = ssd.rms_norm(x, w, held, out=out, residual_out=held)
    assert y2 is out and s2 is held and held._version > v
    assert torch.equal(y, y2) and torch.equal(s, s2)


@pytest.mark.parametrize("fmt", [None, "int8", "e4m3"])
def test_norm_rows_keep_to_themselves(fmt):
    """Infinities, NaN and zeros in a row change no other row, and give what the definition says."""
    x = rn(gen(6), 7, 300).cuda()
    w = torch.ones(300, device="cuda")
    clean = ssd.rms_norm(x, w, format=fmt)
    x[1, 299], x[3, 0], x[5] = INF, NAN, 0
    got = ssd.rms_norm(x, w, format=fmt)
    rows = [0, 2, 4, 6]
    if fmt is None:
        assert torch.equal(got[rows], clean[rows]) and got[[1, 3]].isnan()[:, [299, 0]].any(1).all() and (got[5] == 0).all()
    else:
        assert torch.equal(got[0].float()[rows], clean[0].float()[rows]) and torch.equal(got[1][rows], clean[1][rows])
        assert got[1][[1, 3]].isnan().all() and got[1][5] == 0 and (got[0].float()[[1, 3, 5]] == 0).all()


@pytest.mark.parametrize("D", [300, 1000, 2560, 12001])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_norm_codes_of_weights_that_are_no_numbers(fmt, bad, D):
    """Such a weight is in every row, also against a value of 0; a zero row's scale is 0 without one."""
    x, w = rn(gen(7), 5, D).cuda(), torch.ones(D, device="cuda")
    x[2], x[3, D - 1] = 0, 0
    assert ssd.rms_norm(x, w, format=fmt)[1].isfinite().all()
    w[D - 1] = bad
    codes, scales = ssd.rms_norm(x, w, format=fmt)
    assert scales.isnan().all() and (codes.float() == 0).all()


def test_norm_backward_padding_bits():
    """The sum of the gradients takes the rows as they are; one NaN row leaves the others' dx."""
    g = gen(8)
    x, dout, w = rn(g, 70, 90).cuda(), rn(g, 70, 90).cuda(), torch.ones(90, device="cuda")
    clean = ssd.rms_norm_backward(dout, x, w)
    dout[3, 5] = NAN
    got = ssd.rms_norm_backward(dout, x, w)
    keep = torch.arange(70, device="cuda") != 3
    assert torch.equal(got.dx[keep], clean.dx[keep]) and got.dx[3].isnan().all()


# ---- matrix product -------------------------------------------------------------------------------
LINEAR = [
    # (lead, K, N, type, out type, bias, residual, activation, strided)
    ((1,), 1, 1, "f32", "f32", True, True, None, False),
    ((1,), 2560, 771, "bf16", "bf16", False, False, None, False),
    ((3,), 40, 130, "f16", "f16", True, False, "silu", True),
    ((2, 9), 77, 33, "bf16", "f32", True, True, "gelu", True),
    ((16,), 512, 256, "f16", "f32", False, True, None, False),
    ((33,), 1000, 65, "f32", "f32", True, True, "gelu", False),
    ((64,), 192, 1024, "f16", "f16", True, True, "silu", False),
    ((130,), 8, 257, "bf16", "bf16", False, False, None, False),
    ((257,), 136, 129, "f32", "f32", False, True, "silu", True),
    ((200,), 2049, 300, "bf16", "bf16", True, False, None, True),
    ((300,), 640, 520, "f16", "f16", False, True, None, True),
    ((520,), 320, 1030, "bf16", "bf16", True, True, "silu", False),
    ((7,), 3000, 5, "f16", "f32", False, False, None, False),
    ((1100,), 520, 2500, "bf16", "bf16", True, False, "gelu", False),
]


def linear_case(case, seed):
    lead, K, N, dtype, out, bias, res, act, stride = case
    g, t = gen(seed), DT[dtype]
    x, w = rn(g, *lead, K).to(t), (rn(g, N, K) / K ** 0.5).to(t)
    b = rn(g, N) if bias else None
    r = rn(g, *lead, N).to(DT[out]) if res else None
    view = cuda
    if stride:
        view = lambda v: strided(v.cuda()) if v.dim() > 2 else strided(v[:, None].cuda()).squeeze(1)  # noqa: E731
    return x, w, b, r, view(x), None if r is None else view(r)


def check_product(got, pre, K, S, case, r, name="linear", exact_sums=False):
    out, act = DT[case[4]], case[7]
    want = ref.act(pre, act)
    scale = 1.2 * S + want.abs()
    n = (0 if exact_sums else 2 * K) + 20 + (60 if act else 0)
    if r is not None:
        want, scale = want + r.double(), scale + r.double().abs()
    ref.close(got, want, scale, n, out, name)


@pytest.mark.parametrize("case", LINEAR, ids=str)
def test_linear(case):
    say("linear", case)
    lead, K, N, dtype, out, bias, res, act, _ = case
    x, w, b, r, xg, rg = linear_case(case, 41)
    got, pre = ssd.linear(xg, w.cuda(), cuda(b), rg, activation=act, out_dtype=DT[out], save_pre=True)
    again = ssd.linear(xg, w.cuda(), cuda(b), rg, activation=act, out_dtype=DT[out])
    torch.cuda.synchronize()
    assert got.shape == lead + (N,) and torch.equal(got, again)
    want = ref.product(x, w, b)
    S = ref.product(x, w, b, absolute=True)
    ref.close(pre, want, S, 2 * K + 20, DT[out], "pre")
    check_product(got, want, K, S, case, r)


@pytest.mark.parametrize("case", LINEAR, ids=str)
def test_linear_backward(case):
    say("linear backward", case)
    lead, K, N, dtype, _, bias, _, act, _ = case
    x, w, b, _, xg, _ = linear_case(case, 42)
    g, t = gen(43), DT[dtype]
    dout, pre = rn(g, *lead, N).to(t), rn(g, *lead, N).to(t) if act else None
    kw = dict(pre=cuda(pre), activation=act)
    a, c = (ssd.linear_backward(dout.cuda(), xg, w.cuda(), with_bias=True, **kw) for _ in range(2))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, c))  # a fixed order of summation
    want = ref.product_grads(dout, x, w, pre, act)
    S = ref.product_grads(dout, x, w, pre, act, absolute=True)
    M = x[..., 0].numel()
    half = torch.finfo(t).eps / 2 / ref.U if act else 0  # dpre's own rounding
    ref.close(a.dx.reshape(M, K), want[0], S[0], 2 * N + 80 + half, t, "dx")
    ref.close(a.dweight, want[1], S[1], 2 * M + 80 + half, t, "dweight")
    ref.close(a.dbias, want[2], S[2], M + 80, torch.float32, "dbias")
    only = ssd.linear_backward(dout.cuda(), xg, w.cuda(), with_dx=False, with_dweight=False, with_bias=True, **kw)
    assert only.dx is None and only.dweight is None and torch.equal(only.dbias, a.dbias)
    only = ssd.linear_backward(dout.cuda(), xg, w.cuda(), with_dweight=False, **kw)
    assert only.dbias is None and torch.equal(only.dx, a.dx)
    only = ssd.linear_backward(dout.cuda(), xg, w.cuda(), with_dx=False, **kw)
    assert only.dx is None and torch.equal(only.dweight, a.dweight)


@pytest.mark.parametrize("M,K,N,dtype", [(2100, 520, 1300, "f16"), (300, 1030, 4100, "bf16"), (4099, 257, 130, "bf16"),
                                         (1030, 390, 771, "f32"), (3, 1044, 2514, "f16"), (2514, 1044, 3, "bf16")], ids=str)
def test_linear_backward_of_unlike_contractions(M, K, N, dtype):
    """Both products in one launch or two, their contractions (N and M) of other lengths, alone and together."""
    say("linear backward", M, K, N, dtype)
    g, t = gen(44), DT[dtype]
    x, w, dout = rn(g, M, K).to(t), (rn(g, N, K) / K**0.5).to(t), rn(g, M, N).to(t)
    pre = rn(g, M, N).to(t)
    a = ssd.linear_backward(dout.cuda(), x.cuda(), w.cuda(), with_bias=True, pre=pre.cuda(), activation="silu")
    torch.cuda.synchronize()
    want = ref.product_grads(dout, x, w, pre, "silu")
    S = ref.product_grads(dout, x, w, pre, "silu", absolute=True)
    half = torch.finfo(t).eps / 2 / ref.U  # dpre's own rounding
    for got, exact, size, n, out, name in zip(a, want, S, (2 * N + 80 + half, 2 * M + 80 + half, M + 80), (t, t, torch.float32),
                                              ("dx", "dweight", "dbias")):
        ref.close(got, exact, size, n, out, name)
        alone = ssd.linear_backward(dout.cuda(), x.cuda(), w.cuda(), pre=pre.cuda(), activation="silu", with_dx=name == "dx",
                                    with_dweight=name == "dweight", with_bias=name == "dbias")
        ref.close(getattr(alone, name), exact, size, n, out, name)


@pytest.mark.parametrize("shift,gap", [(4, 8), (16, 4), (2, 2), (0, 16)], ids=str)
@pytest.mark.parametrize("M,K,N,dtype", [(1, 2562, 300, "bf16"), (16, 1110, 771, "f32"), (70, 302, 130, "f16"), (1, 1, 1, "f32"),
                                         (33, 1540, 771, "int8"), (5, 260, 64, "e4m3"), (129, 2, 33, "bf16"),
                                         (600, 1002, 700, "bf16")], ids=str)
def test_linear_of_rows_between_16_bytes(M, K, N, dtype, shift, gap):
    """Rows of a multiple of 4 bytes (and ones that are not, by their stride or first byte), among values that would show."""
    g = gen(45)
    if dtype in DT:
        t = DT[dtype]
        x, w = rn(g, M, K).to(t), (rn(g, N, K) / K**0.5).to(t)
    elif dtype == "int8":
        t = torch.int8
        x, w = (torch.randint(-128, 128, s, generator=g, dtype=t) for s in ((M, K), (N, K)))
    else:
        t = torch.float8_e4m3fn
        x, w = ((100 * rn(g, *s)).clamp(-448, 448).to(t) for s in ((M, K), (N, K)))
    shift, gap = -(-shift // t.itemsize), -(-gap // t.itemsize)
    flat = torch.full((M * (K + gap) * t.itemsize + 64,), 0x7f, dtype=torch.uint8, device="cuda")  # (fp16, e4m3: NaN)
    if dtype in ("bf16", "f32"):
        flat.fill_(0xff)  # NaN
    rows = flat.view(t)[shift:shift + M * (K + gap)].view(M, K + gap)[:, :K]
    rows.view(torch.uint8).copy_(x.cuda().view(torch.uint8))
    tail = torch.full((N * K * t.itemsize + 64,), 0xff if dtype in ("bf16", "f32") else 0x7f, dtype=torch.uint8, device="cuda")
    wg = tail.view(t)[:N * K].view(N, K)
    wg.view(torch.uint8).copy_(w.cuda().view(torch.uint8))
    got = ssd.linear(rows, wg, out_dtype=torch.float32)
    torch.cuda.synchronize()
    want, S = (ref.product(x, w, None, None, None, absolute=k) for k in (False, True))
    ref.close(got, want, S, (0 if dtype == "int8" else 2 * K) + 20, torch.float32, "linear")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "int8", "e4m3"])
@pytest.mark.parametrize("M,K,N,shift", [(1, 64, 70, 1), (1, 64, 70, 3), (1, 2560, 300, 5), (2, 64, 70, 1), (200, 192, 130, 7),
                                         (1, 64, 70, 16)], ids=str)
def test_linear_of_contiguous_rows_that_start_anywhere(M, K, N, shift, dtype):
    """A slice of one row, and rows behind an odd offset, both contiguous: the bits of the same values on a border."""
    say("contiguous rows", M, K, N, shift, dtype)
    g = gen(46)
    if dtype in DT:
        wide, w = rn(g, M * K + 16).to(DT[dtype]).cuda(), (rn(g, N, K) / K**0.5).to(DT[dtype]).cuda()
    else:
        wide, w = (torch.randint(-100, 100, s, generator=g, dtype=torch.int8).cuda() for s in ((M * K + 16,), (N, K)))
        if dtype == "e4m3":
            wide, w = wide.float().to(torch.float8_e4m3fn), w.float().to(torch.float8_e4m3fn)
    x = wide[None, shift:shift + K] if M == 1 else wide[shift:shift + M * K].view(M, K)
    assert x.is_contiguous() and x.data_ptr() % 16 == shift * x.element_size() % 16
    aligned = torch.empty_like(x).copy_(x)
    want = ssd.linear(aligned, w, out_dtype=torch.float32)
    for _ in range(2):
        assert torch.equal(ssd.linear(x, w, out_dtype=torch.float32), want)
        assert torch.equal(ssd.linear(aligned, w, out_dtype=torch.float32), want)
    pre, S = (ref.product(aligned.cpu(), w.cpu(), absolute=k) for k in (False, True))
    ref.close(want, pre, S, 2 * K + 20, torch.float32, "linear")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "int8", "e4m3"])
@pytest.mark.parametrize("M,K,N,first", [(1, 77, 70, 1), (3, 1541, 130, 3), (200, 259, 300, 5), (1, 1542, 70, 3), (5, 70, 64, 1),
                                         (300, 1002, 520, 7)], ids=str)
def test_linear_with_rows_cut_out_of_a_joint_weight(M, K, N, first, dtype):
    """Part of a weight whose rows are no multiple of 16 bytes: the bits of a weight of its own."""
    say("part of a weight", M, K, N, first, dtype)
    g = gen(47)
    if dtype in DT:
        x, joint = rn(g, M, K).to(DT[dtype]).cuda(), (rn(g, N + first + 2, K) / K**0.5).to(DT[dtype]).cuda()
    else:
        x, joint = (torch.randint(-100, 100, s, generator=g, dtype=torch.int8).cuda() for s in ((M, K), (N + first + 2, K)))
        if dtype == "e4m3":
            x, joint = x.float().to(torch.float8_e4m3fn), joint.float().to(torch.float8_e4m3fn)
    joint[:first], joint[first + N:] = (NAN, NAN) if dtype != "int8" else (127, 127)
    w = joint[first:first + N]
    got = ssd.linear(x, w, out_dtype=torch.float32)
    assert torch.equal(got, ssd.linear(x, torch.empty_like(w).copy_(w), out_dtype=torch.float32))
    pre, S = (ref.product(x.cpu(), w.cpu(), absolute=k) for k in (False, True))
    ref.close(got, pre, S, 2 * K + 20, torch.float32, "linear")


CODES = [
    # (lead, K, N, type, out type, bias, residual, activation, strided, scales)
    ((1,), 16, 8, "int8", "f32", False, False, None, False, True),
    ((5,), 300, 77, "int8", "bf16", True, True, "silu", False, True),
    ((33,), 1536, 771, "int8", "f16", False, False, None, False, True),
    ((200,), 640, 300, "int8", "f32", True, False, None, True, False),
    ((1,), 2560, 100, "e4m3", "bf16", False, False, None, False, True),
    ((2, 20), 129, 260, "e4m3", "f32", True, True, "gelu", True, True),
    ((300,), 2000, 513, "e4m3", "f16", False, True, None, False, True),
    ((70,), 128, 64, "e4m3", "f32", False, False, None, False, False),
]


@pytest.mark.parametrize("case", CODES, ids=str)
def test_linear_of_codes(case):
    say("linear of codes", case)
    lead, K, N, fmt, out, bias, res, act, stride, scales = case
    g = gen(44)
    if fmt == "int8":
        x, w = (torch.randint(-128, 128, s, generator=g, dtype=torch.int8) for s in (lead + (K,), (N, K)))
        x[..., 0], w[:, 0] = -128, -128
    else:
        x, w = ((100 * rn(g, *s)).clamp(-448, 448).to(torch.float8_e4m3fn) for s in (lead + (K,), (N, K)))
    sx, sw = (torch.exp(rn(g, *lead)) / 1000, torch.exp(rn(g, N)) / 100) if scales else (None, None)
    b, r = rn(g, N) if bias else None, rn(g, *lead, N).to(DT[out]) if res else None
    xg = x.cuda()
    if stride:
        wide = torch.zeros(lead + (K + 5,), dtype=torch.int8, device="cuda")
        wide[..., 3:3 + K] = xg.view(torch.int8)
        xg = wide[..., 3:3 + K].view(x.dtype)
    got = ssd.linear(xg, w.cuda(), cuda(b), cuda(r), activation=act, x_scale=cuda(sx), weight_scale=cuda(sw),
                     out_dtype=DT[out])
    torch.cuda.synchronize()
    pre, S = (ref.product(x, w, b, sx, sw, absolute=k) for k in (False, True))
    check_product(got, pre, K, S, case, r, exact_sums=fmt == "int8")


@pytest.mark.parametrize("M,K,N", [(64, 8, 64), (64, 32, 64), (16, 64, 64), (5, 129, 70), (300, 2560, 1000), (2048, 256, 10576)])
def test_e4m3_sums_in_fp32(M, K, N):
    """Outputs in fp32 are within two roundings a product, also where there are few and of unlike size."""
    g = torch.Generator(device="cuda").manual_seed(48)
    x, w = ((100 * torch.randn(*s, generator=g, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn) for s in ((M, K), (N, K)))
    got = ssd.linear(x, w, out_dtype=torch.float32).double()
    a, b = x.float().double(), w.float().double()
    want, S = a @ b.t(), a.abs() @ b.t().abs()
    assert ((got - want).abs() <= (2 * K + 20) * ref.U * S).all()


def test_e4m3_products_of_unlike_size():
    """Codes times one beside 2^16, in each of 16 places: sums of 24 bits, exact in fp32."""
    values = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).float()
    values = values[values.isfinite() & (values.abs() >= 2.0**-4)]  # multiples of 2^-7: 2^16 and that have 24 bits
    one = torch.zeros(len(values), 40, device="cuda")
    one[:, 3] = 256
    for k in range(16):
        x = one.clone()
        x[:, 4 + k] = values
        w = torch.zeros(1, 40, device="cuda")
        w[0, 3], w[0, 4 + k] = 256, 1
        got = ssd.linear(x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn), out_dtype=torch.float32)[:, 0]
        assert torch.equal(got.double(), 65536 + values.double()), k


def test_int8_sums_are_exact():
    """The widest contraction of the largest codes: 2^31 less 2^14."""
    K = 131071
    x = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    got = ssd.linear(x, w, out_dtype=torch.float32)
    assert (got == float((1 << 31) - (1 << 14))).all()


@pytest.mark.parametrize("M,K,N", [(5, 40, 7), (130, 72, 140), (300, 1000, 300)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_linear_rows_keep_to_themselves(M, K, N, dtype):
    """A NaN row of x or weight gives NaN in its own row or column and changes no other; neither do values around a view."""
    g, t = gen(9), DT[dtype]
    x, w = rn(g, M, K).to(t).cuda(), rn(g, N, K).to(t).cuda()
    clean = ssd.linear(x, w)
    assert torch.equal(ssd.linear(strided(x[:, None]).squeeze(1), w), clean)
    x[M - 1, K - 1], w[N - 1, 0] = NAN, INF
    got = ssd.linear(x, w)
    assert torch.equal(got[:-1, :-1], clean[:-1, :-1]) and got[-1].isnan().all() and not got[:-1, -1].isfinite().any()


@pytest.mark.parametrize("M,N", [(3, 40), (200, 333), (300, 1024)])
def test_linear_onto_the_residual_in_place(M, N):
    g = gen(10)
    x, w, r = rn(g, M, 512).bfloat16().cuda(), rn(g, N, 512).bfloat16().cuda(), rn(g, M, N).bfloat16().cuda()
    want = ssd.linear(x, w, residual=r, activation="silu")
    v = r._version
    got = ssd.linear(x, w, residual=r, activation="silu", out=r)
    assert got is r and r._version > v and torch.equal(got, want)


def test_nan_codes_and_scales_stay_in_their_rows():
    x = torch.ones(5, 256, device="cuda").to(torch.float8_e4m3fn)
    w = torch.ones(70, 256, device="cuda").to(torch.float8_e4m3fn)
    s = torch.ones(5, device="cuda")
    x.view(torch.uint8)[1, 200], s[3] = 0x7f, NAN
    w.view(torch.uint8)[7, 0] = 0xff
    got = ssd.linear(x, w, x_scale=s, out_dtype=torch.float32)
    bad = torch.zeros(5, 70, dtype=torch.bool, device="cuda")
    bad[[1, 3]], bad[:, 7] = True, True
    assert torch.equal(got.isnan(), bad) and (got[~bad] == 256).all()


@pytest.mark.parametrize("act,want", [("silu", [0.0, INF, 0.0]), ("gelu", [0.0, INF, 0.0])])
def test_activations_of_infinities(act, want):
    x, w = torch.ones(1, 1, device="cuda"), torch.tensor([[-INF], [INF], [0.0]], device="cuda")
    assert ssd.linear(x, w, activation=act)[0].tolist() == want
    pre = torch.tensor([[-INF, INF, -200.0, 200.0, 0.0]], device="cuda")
    g = ssd.linear_backward(torch.ones(1, 5, device="cuda"), x, torch.ones(5, 1, device="cuda"), pre=pre, activation=act)
    assert g.dweight[:, 0].tolist() == [0.0, 1.0, 0.0, 1.0, 0.5]


# ---- gated recurrence -------------------------------------------------------------------------------
REC = [
    # (B, L, D, dtype, state type, packing, initial state, in_gate, biases, normalize, strided)
    (1, 1, 1, "f32", "f32", None, True, True, True, True, False),
    (2, 3, 5, "bf16", "f32", None, True, True, True, True, False),
    (1, 127, 64, "f16", "f16", None, False, True, False, True, False),
    (2, 128, 33, "bf16", "bf16", None, True, False, True, False, True),
    (1, 129, 130, "f32", "f32", None, True, True, True, True, True),
    (3, 300, 34, "f16", "f32", "pad", True, True, True, True, True),
    (2, 260, 31, "f32", "f16", "full", True, False, False, True, False),
    (2, 40, 24, "f32", "f32", "ones", True, True, True, False, False),
    (1, 1000, 7, "bf16", "f32", "pad", False, True, True, True, False),
    (1, 4500, 40, "f16", "f32", None, True, True, True, True, False),
    (1, 2100, 34, "bf16", "f32", "pad", True, True, True, True, True),
    (40, 150, 250, "bf16", "f32", None, True, True, True, True, False),
    (1, 5000, 200, "f32", "f32", "pad", True, True, True, True, False),
]


def rec_case(case, seed):
    B, L, D, dtype, st, pack, state, gated, biases, normalize, stride = case
    g, t = gen(seed), DT[dtype]
    seq, S = packing(B, L, pack, g)
    x, gate = rn(g, B, L, D).to(t), (2 * rn(g, B, L, D)).to(t)
    ig = (2 * rn(g, B, L, D)).to(t) if gated else None
    A = -torch.exp(rn(g, D) - 2).clamp(max=2.0)
    gb, ib = rn(g, D) if biases else None, rn(g, D) if biases and gated else None
    h0 = rn(g, S, D).to(DT[st]) if state else None
    view = (lambda v: strided(v.cuda())) if stride else cuda  # noqa: E731
    args = [view(x), view(gate), A.cuda(), None if ig is None else view(ig), cuda(gb), cuda(ib)]
    kw = dict(normalize=normalize, seq_idx=cuda(seq), nseq=S if pack else None, initial_state=cuda(h0), state_dtype=DT[st])
    return (x, gate, A, ig, gb, ib), h0, seq, S, args, kw, g


def per_token(A):
    return 14 + 14 * float(A.abs().max())


@pytest.mark.parametrize("case", REC, ids=str)
def test_recurrence(case):
    say("recurrence", case)
    B, L, D, dtype, st, *_ = case
    ins, h0, seq, S, args, kw, _ = rec_case(case, 51)
    out, fin = ssd.gated_recurrence(*args, **kw)
    torch.cuda.synchronize()
    rr = ref.runs(B, L, seq)
    want, wfin, _ = ref.recurrence(*ins, case[9], h0, S, rr)
    scale, sfin, _ = ref.recurrence(*ins, case[9], h0, S, rr, absolute=True)
    K = L * per_token(ins[2]) + 100
    ref.close(out, want, scale, K, ins[0].dtype, "out")
    ref.close(fin, wfin, sfin, K, DT[st], "final state")
    assert torch.equal(ssd.gated_recurrence(*args, **kw, with_final_state=False)[0], out)


def used(t, seq, S):
    if seq is None:
        return t
    return torch.where(((seq >= 0) & (seq < S))[..., None], t, torch.zeros((), dtype=t.dtype))


@pytest.mark.parametrize("case", REC, ids=str)
def test_recurrence_backward(case):
    say("recurrence backward", case)
    B, L, D, dtype, st, *_ = case
    ins, h0, seq, S, args, kw, g = rec_case(case, 52)
    dout, dfin = rn(g, B, L, D).to(ins[0].dtype), rn(g, S, D).to(DT[st])
    out, _, saved = ssd.gated_recurrence(*args, **kw, save_for_backward=True)
    a, b = (ssd.gated_recurrence_backward(dout.cuda(), *args, saved=saved, dfinal_state=dfin.cuda(), **kw) for _ in range(2))
    torch.cuda.synchronize()
    for p, q in zip(a, b):
        assert (p is None and q is None) or torch.equal(p, q)  # a fixed order of summation
    rr = ref.runs(B, L, seq)
    dout = used(dout, seq, S)
    want = ref.recurrence_grads(dout, dfin, *ins, case[9], h0, S, rr)
    scale = ref.recurrence_grads(dout, dfin, *ins, case[9], h0, S, rr, absolute=True)
    K, t, f = 2 * L * per_token(ins[2]) + 200, ins[0].dtype, torch.float32
    names = ("dx", "dgate", "dA", "din_gate", "dgate_bias", "din_bias", "dh0")
    for i, (v, ty, k) in enumerate(zip(a, (t, t, f, t, f, f, DT[st]), (0, 0, B * L, 0, B * L, B * L, 0))):
        given = (ins[0], ins[1], ins[2], ins[3], ins[4], ins[5], h0)[i]
        assert (v is None) == (given is None)
        if v is not None:
            ref.close(v, want[i], scale[i], K + k, ty, names[i])
    if seq is not None:  # padding gets zero gradients
        pad = ((seq < 0) | (seq >= S)).cuda()
        assert (a.dx[pad] == 0).all() and (a.dgate[pad] == 0).all()


def test_recurrence_padding_may_hold_anything():
    case = (2, 300, 34, "f32", "f32", "pad", True, True, True, True, False)
    ins, h0, seq, S, args, kw, g = rec_case(case, 53)
    pad = (seq < 0).cuda()
    dout = rn(g, 2, 300, 34).cuda()
    out, fin, saved = ssd.gated_recurrence(*args, **kw, save_for_backward=True)
    a = ssd.gated_recurrence_backward(dout, *args, saved=saved, **kw)
    for t in (args[0], args[1], args[3], dout):
        t[pad] = NAN
    out2, fin2, saved2 = ssd.gated_recurrence(*args, **kw, save_for_backward=True)
    b = ssd.gated_recurrence_backward(dout, *args, saved=saved2, **kw)
    assert torch.equal(out[~pad], out2[~pad]) and torch.equal(fin, fin2)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_recurrence_sequences_keep_to_themselves():
    """A NaN in one sequence stays there, forward and backward, across tiles and time splits."""
    case = (1, 2100, 34, "f32", "f32", "full", True, True, True, True, False)
    ins, h0, seq, S, args, kw, g = rec_case(case, 54)
    dout = rn(g, 1, 2100, 34).cuda()
    _, _, saved = ssd.gated_recurrence(*args, **kw, save_for_backward=True)
    out, fin = ssd.gated_recurrence(*args, **kw)
    a = ssd.gated_recurrence_backward(dout, *args, saved=saved, **kw)
    q = int(seq[0, 1000])
    args[0][0, 1000, 3] = NAN
    out2, fin2, saved2 = ssd.gated_recurrence(*args, **kw, save_for_backward=True)
    b = ssd.gated_recurrence_backward(dout, *args, saved=saved2, **kw)
    other = (seq[0] != q).cuda()
    assert torch.equal(out[0, other], out2[0, other]) and out2[0, 1000, 3].isnan()
    keep = torch.arange(S) != q
    assert torch.equal(fin[keep.cuda()], fin2[keep.cuda()]) and fin2[q, 3].isnan()
    assert torch.equal(a.dx[0, other], b.dx[0, other]) and torch.equal(a.dgate[0, other], b.dgate[0, other])


@pytest.mark.parametrize("A,gate", [(0.0, 0.0), (-INF, 0.0), (-1.0, -INF), (-1.0, INF), (-1e30, -200.0), (-0.01, -90.0)])
@pytest.mark.parametrize("packed", [False, True])
def test_recurrence_extreme_decays(A, gate, packed):
    """No decay, nothing kept, closed and open gates: finite values, the definition's; a closed gate's gradient counts as 0."""
    B, L, D = 1, 140, 4
    g = gen(55)
    x, gt = rn(g, B, L, D), torch.full((B, L, D), gate)
    Av, h0 = torch.full((D,), A), rn(g, B, D)
    seq = torch.zeros(B, L, dtype=torch.int32) if packed else None
    kw = dict(initial_state=h0.cuda(), seq_idx=cuda(seq), nseq=1 if packed else None)
    args = (x.cuda(), gt.cuda(), Av.cuda())
    out, fin, saved = ssd.gated_recurrence(*args, save_for_backward=True, **kw)
    want, wfin, _ = ref.recurrence(x, gt, Av, None, None, None, True, h0, 1, [(0, 0, 0, L)])
    scale, _, _ = ref.recurrence(x, gt, Av, None, None, None, True, h0, 1, [(0, 0, 0, L)], absolute=True)
    ref.close(out, want, scale + 1, L * 28 + 100, torch.float32, "out")
    ref.close(fin, wfin, scale[:, -1] + 1, L * 28 + 100, torch.float32, "final state")
    got = ssd.gated_recurrence_backward(torch.ones(B, L, D, device="cuda"), *args, saved=saved, **kw)
    assert all(v is None or v.isfinite().all() for v in got)


@pytest.mark.parametrize("dtype,st,D,B,slots,gated", [("bf16", "f32", 70, 5, 9, True), ("f32", "bf16", 64, 1, 1, False),
                                                      ("f16", "f16", 5, 3, 3, True), ("bf16", "f32", 2564, 33, 40, True)])
def test_recurrence_step_continues_the_prompt(dtype, st, D, B, slots, gated):
    say("recurrence step", dtype, st, D, B, slots)
    g, t = gen(56), DT[dtype]
    L = 9
    x, gate, ig = (rn(g, B, L, D).to(t) for _ in range(3))
    ig = ig if gated else None
    A, gb, ib = -torch.exp(rn(g, D) - 2), rn(g, D), rn(g, D) if gated else None
    pool = rn(g, slots, D).to(DT[st])
    index = torch.randperm(slots, generator=g)[:B].to(torch.int32)
    held = pool.clone().cuda()
    v = held._version
    h = pool[index.long()].double()
    K = per_token(A) + 100
    for k in range(L):
        wide = lambda z: None if z is None else strided(z[:, k:k + 1].cuda()).squeeze(1)  # noqa: E731
        h0 = held[index.long().cuda()].cpu()
        got = ssd.gated_recurrence_step(wide(x), wide(gate), A.cuda(), wide(ig), gb.cuda(), cuda(ib), state=held,
                                        slots=index.cuda())
        one = slice(k, k + 1)
        ins = (x[:, one], gate[:, one], A, None if ig is None else ig[:, one], gb, ib)
        rr = ref.runs(B, 1)
        want, wfin, _ = ref.recurrence(*ins, True, h0, B, rr)
        S, _, _ = ref.recurrence(*ins, True, h0, B, rr, absolute=True)
        ref.close(got, want[:, 0], S[:, 0], K, t, "out")
        ref.close(held[index.long().cuda()], wfin, S[:, 0], K, DT[st], "state")
    assert held._version > v
    rest = torch.ones(slots, dtype=torch.bool)
    rest[index.long()] = False
    assert torch.equal(held.cpu()[rest], pool[rest])


def test_recurrence_step_of_padded_batches():
    g = gen(57)
    x, gate, A = rn(g, 4, 6).cuda(), rn(g, 4, 6).cuda(), -torch.ones(6, device="cuda")
    pool = rn(g, 3, 6).cuda()
    before = pool.clone()
    out = ssd.gated_recurrence_step(x, gate, A, state=pool, slots=torch.tensor([2, -1, 3, 0], dtype=torch.int32).cuda())
    assert (out[[1, 2]] == 0).all() and torch.equal(pool[1], before[1]) and not torch.equal(pool[2], before[2])
    same = before.clone()
    direct = ssd.gated_recurrence_step(x[[0]], gate[[0]], A, state=same[2:3])
    assert torch.equal(direct[0], out[0]) and torch.equal(same[2], pool[2])


def test_recurrence_prompt_in_two_pieces():
    g = gen(58)
    x, gate, ig = (rn(g, 2, 700, 50).cuda() for _ in range(3))
    A = -torch.exp(rn(g, 50) - 2).cuda()
    whole, fin = ssd.gated_recurrence(x, gate, A, ig)
    a, mid = ssd.gated_recurrence(
        x[:, :333].contiguous(), gate[:, :333].contiguous(), A, ig[:, :333].contiguous())
    b, end = ssd.gated_recurrence(x[:, 333:].contiguous(), gate[:, 333:].contiguous(), A, ig[:, 333:].contiguous(),
                                  initial_state=mid)
    S = ref.recurrence(x, gate, A, ig, None, None, True, None, 2, ref.runs(2, 700), absolute=True)
    K = 2 * (700 * per_token(A) + 100)  # both sides are off by that at most
    ref.close(torch.cat([a, b], 1), whole, S[0], K, torch.float32, "out")
    ref.close(end, fin, S[1], K, torch.float32, "state")


# ---- sizes past 32 bits -----------------------------------------------------------------------------
def test_norm_past_32_bits():
    """More than 2^32 bytes and 2^31 values: the last rows are those of a call on them alone."""
    M, D = 140000, 16001
    x = torch.empty(M, D, dtype=torch.float16, device="cuda").normal_()
    w = torch.rand(D, device="cuda")
    y, s = ssd.rms_norm(x, w, x)
    rows = slice(M - 3, M)
    want = ssd.rms_norm(x[rows], w, x[rows])
    assert torch.equal(y[rows], want[0]) and torch.equal(s[rows], want[1])
    codes, scales = ssd.rms_norm(x, w, format="int8")
    want = ssd.rms_norm(x[rows], w, format="int8")
    assert torch.equal(codes[rows], want[0]) and torch.equal(scales[rows], want[1])
    del codes, s
    g = ssd.rms_norm_backward(y, x, w)
    want = ssd.rms_norm_backward(y[rows], x[rows], w)
    assert torch.equal(g.dx[rows], want.dx)


def test_linear_past_32_bits():
    """More than 2^32 bytes of x, of a view of x, and of out."""
    M, K = 600000, 4096
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.empty(70, K, dtype=torch.bfloat16, device="cuda").normal_()
    rows = [0, 1, 262143, 262144, 524287, 524288, M - 1]
    ref64 = x[rows].cpu().double() @ w.cpu().double().t()
    S = x[rows].cpu().double().abs() @ w.cpu().double().abs().t()
    ref.close(ssd.linear(x, w)[rows], ref64, S, 2 * K + 20, torch.bfloat16, "out")
    part = x[:, 3:2003]
    ref64 = part[rows].cpu().double() @ w[:, :2000].cpu().double().t()
    ref.close(ssd.linear(part, w[:, :2000].contiguous())[rows], ref64, S, 2 * K + 20, torch.bfloat16, "out of a view")
    del part
    u, v = x[:, :8].contiguous(), torch.empty(4000, 8, dtype=torch.bfloat16, device="cuda").normal_()
    del x
    out = ssd.linear(u, v)
    ref64, S = u[rows].cpu().double() @ v.cpu().double().t(), u[rows].cpu().double().abs() @ v.cpu().double().abs().t()
    ref.close(out[rows], ref64, S, 36, torch.bfloat16, "wide out")


def test_recurrence_past_32_bits():
    """More than 2^31 values: the last tokens are those of a call that starts from the state before them."""
    L, D, n = 270000, 8100, 301
    x, gate = (torch.empty(1, L, D, device="cuda").normal_() for _ in range(2))
    A = -torch.exp(torch.empty(D, device="cuda").normal_() - 2)
    out, fin, saved = ssd.gated_recurrence(x, gate, A, save_for_backward=True)
    tail = lambda t: t[:, L - n:].contiguous()  # noqa: E731
    want, wfin = ssd.gated_recurrence(tail(x), tail(gate), A, initial_state=out[:, L - n - 1].clone())
    S = ref.recurrence(tail(x), tail(gate), A, None, None, None, True, out[:, L - n - 1], 1, [(0, 0, 0, n)], absolute=True)
    K = 2 * (n * per_token(A) + 100)
    ref.close(tail(out), want, S[0], K, torch.float32, "out")
    ref.close(fin, wfin, S[1], K, torch.float32, "state")
    assert out.isfinite().all()
    del want, gate, saved
    gate = out  # (any values do)
    h = ssd.gated_recurrence(x, gate, A, save_for_backward=True)
    g = ssd.gated_recurrence_backward(x, x, gate, A, saved=h[2])
    w, _, ws = ssd.gated_recurrence(tail(x), tail(gate), A, initial_state=h[0][:, L - n - 1].clone(), save_for_backward=True)
    b = ssd.gated_recurrence_backward(tail(x), tail(x), tail(gate), A, initial_state=h[0][:, L - n - 1].clone(), saved=ws)
    S = ref.recurrence_grads(tail(x), None, tail(x), tail(gate), A, None, None, None, True, h[0][:, L - n - 1], 1, [(0, 0, 0, n)],
                             absolute=True)
    K = 2 * (2 * n * per_token(A) + 200)
    ref.close(tail(g.dx), b.dx, S[0], K, torch.float32, "dx")
    ref.close(tail(g.dgate), b.dgate, S[1], K, torch.float32, "dgate")


def test_recurrence_step_of_far_rows():
    wide = torch.empty(3, 700_000_000, dtype=torch.float16, device="cuda")
    x, gate = wide[:, :70], wide[:, 699_999_900:699_999_970]
    x.normal_()
    gate.normal_()
    A, pool = -torch.ones(70, device="cuda"), torch.ones(3, 70, device="cuda")
    other = pool.clone()
    got = ssd.gated_recurrence_step(x, gate, A, state=pool)
    assert torch.equal(got, ssd.gated_recurrence_step(x.contiguous(), gate.contiguous(), A, state=other))
    assert torch.equal(pool, other)


# ---- together ---------------------------------------------------------------------------------------
def layer_weights(g, D, E, t):
    w = dict(norm=1 + 0.2 * rn(g, D), inp=(rn(g, 3 * E, D) / D ** 0.5).to(t), conv=0.5 * rn(g, E, 4), convb=0.1 * rn(g, E),
             A=torch.log(0.9 + 0.099 * torch.rand(E, generator=g)), gb=rn(g, E), ib=rn(g, E), out=(rn(g, D, E) / E ** 0.5).to(t))
    return {k: v.cuda() for k, v in w.items()}


def layer(x, s, w, E, states=None, save=False):
    """One layer as a program runs it: norm, joint projection, convolution, recurrence, projection onto the stream."""
    y, s = ssd.rms_norm(x, w["norm"], s)
    p = ssd.linear(y, w["inp"])
    u, gate, ig = p[..., :E], p[..., E:2 * E], p[..., 2 * E:]
    if states is not None and x.dim() == 2:
        c = ssd.causal_conv_step(u, w["conv"], w["convb"], state=states[0])
        h = ssd.gated_recurrence_step(c, gate, w["A"], ig, w["gb"], w["ib"], state=states[1])
        return ssd.linear(h, w["out"]), s
    c, cs = ssd.causal_conv(u, w["conv"], w["convb"])
    h, hs, *saved = ssd.gated_recurrence(c, gate, w["A"], ig, w["gb"], w["ib"], save_for_backward=save)
    return ssd.linear(h, w["out"]), s, (cs, hs), (y, u, gate, ig, c, h, *saved)


def plain_layer(x, s, w, E):
    """The same in 64 bits."""
    s = x + s
    y = s / (s.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w["norm"]
    p = y @ w["inp"].t()
    u, gate, ig = p[..., :E], p[..., E:2 * E], p[..., 2 * E:]
    L = x.shape[1]
    up = torch.cat([u.new_zeros(u.shape[0], 3, E), u], 1)
    c = torch.nn.functional.silu(sum(up[:, k:k + L] * w["conv"][:, k] for k in range(4)) + w["convb"])
    lo = w["A"] * torch.sigmoid(gate + w["gb"])
    a, add = torch.exp(lo), torch.sqrt(-torch.expm1(2 * lo)) * torch.sigmoid(ig + w["ib"]) * c
    h, hs = torch.zeros_like(c[:, 0]), []
    for t in range(L):
        h = a[:, t] * h + add[:, t]
        hs.append(h)
    return torch.stack(hs, 1) @ w["out"].t(), s


def test_a_layer_over_a_prompt_then_token_by_token():
    """The operators in the order that a model calls them; fp32, so that the bound is that of its sums: 2 K for each of the
    two products and a token's roundings over the sequence, of values of size 1 to 4."""
    B, L, D, E = 2, 150, 96, 160
    g = gen(61)
    w = layer_weights(g, D, E, torch.float32)
    x, s = rn(g, B, L, D), rn(g, B, L, D)
    want, wsum = plain_layer(x.double(), s.double(), {k: v.cpu().double() for k, v in w.items()}, E)
    n = 130
    out, total, states, _ = layer(x[:, :n].cuda(), s[:, :n].cuda(), w, E)
    outs, sums = [out], [total]
    for t in range(n, L):
        o, ts = layer(x[:, t].cuda(), s[:, t].cuda(), w, E, states)
        outs.append(o[:, None])
        sums.append(ts[:, None])
    got = torch.cat(outs, 1).cpu().double()
    assert torch.equal(torch.cat(sums, 1).cpu(), x + s)
    tol = ref.U * (2 * D + 2 * E + 28 * 40 + 200) * 4 * float(want.abs().max())  # a state forgets within some 40 tokens
    assert float((got - want).abs().max()) < tol


def test_a_layer_s_gradients():
    """Forward and backward calls of one layer against autograd through the 64-bit form."""
    B, L, D, E = 2, 140, 40, 48
    g = gen(62)
    w = layer_weights(g, D, E, torch.float32)
    x, s, dout, dsum = (rn(g, B, L, D) for _ in range(4))
    _, total, _, (y, u, gate, ig, c, h, saved) = layer(x.cuda(), s.cuda(), w, E, save=True)
    go = ssd.linear_backward(dout.cuda(), h, w["out"])
    gr = ssd.gated_recurrence_backward(go.dx, c, gate, w["A"], ig, w["gb"], w["ib"], saved=saved)
    gc = ssd.causal_conv_backward(gr.dx, u, w["conv"], w["convb"])
    gi = ssd.linear_backward(torch.cat([gc.dx, gr.dgate, gr.din_gate], -1), y, w["inp"])
    gn = ssd.rms_norm_backward(gi.dx, total, w["norm"], dresidual=dsum.cuda())
    got = dict(x=gn.dx, s=gn.dresidual, norm=gn.dweight, inp=gi.dweight, conv=gc.dweight, convb=gc.dbias, A=gr.dA,
               gb=gr.dgate_bias, ib=gr.din_bias, out=go.dweight)
    w64 = {k: v.cpu().double().requires_grad_() for k, v in w.items()}
    x64, s64 = x.double().requires_grad_(), s.double().requires_grad_()
    o, t = plain_layer(x64, s64, w64, E)
    ((o * dout.double()).sum() + (t * dsum.double()).sum()).backward()
    want = dict(x=x64.grad, s=s64.grad, **{k: v.grad for k, v in w64.items()})
    for k, v in got.items():
        # in the 2-norm: relative to the whole gradient, with the roundings of the forward and the backward chain
        off = float((v.cpu().double() - want[k]).norm() / want[k].norm())
        assert off < ref.U * 8 * (2 * D + 2 * E + 28 * 40 + 200), (k, off)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_norm_and_product_in_8_bits(fmt):
    """Codes and scales go from the norm into the product as they are."""
    g = gen(63)
    x, r, w = rn(g, 37, 200).bfloat16(), rn(g, 37, 200).bfloat16(), 1 + 0.2 * rn(g, 200)
    wc = torch.randint(-127, 128, (90, 200), generator=g, dtype=torch.int8) if fmt == "int8" else rn(g, 90, 200).to(torch.float8_e4m3fn)
    ws = torch.exp(rn(g, 90)) / 100
    codes, scales, s = ssd.rms_norm(x.cuda(), w.cuda(), r.cuda(), format=fmt)
    out = ssd.linear(codes, wc.cuda(), x_scale=scales, weight_scale=ws.cuda(), out_dtype=torch.float32)
    pre, S = (ref.product(codes.cpu(), wc, None, scales.cpu(), ws, absolute=k) for k in (False, True))
    ref.close(out, pre, S, 2 * 200 + 20, torch.float32, "out")
    # against the product without codes: each value is off by half a code's step at most
    _, y = ref.norm(x, r, w, 1e-5)
    step = ref.code_step(y / scales.cpu().double()[:, None], fmt) * scales.cpu().double()[:, None] / 2
    wv = wc.float().double() * ws.double()[:, None]
    bound = step @ wv.abs().t() * 1.01 + 1e-4
    assert ((out.cpu().double() - y @ wv.t()).abs() <= bound).all()


# ---- how they are called ------------------------------------------------------------------------------
def some_calls(g):
    """(name, call, its tensors) of every entry point, on small inputs; a call makes its outputs anew from clones."""
    x, r, w = rn(g, 3, 70, 40).cuda(), rn(g, 3, 70, 40).cuda(), rn(g, 40).cuda()
    W, A, pool = rn(g, 24, 40).cuda(), -torch.exp(rn(g, 40)).cuda(), rn(g, 70, 40).cuda()
    dy = rn(g, 3, 70, 24).cuda()
    saved = ssd.gated_recurrence(x, r, A, save_for_backward=True)[2]

    def step():
        p = pool.clone()
        return ssd.gated_recurrence_step(x[0], r[0], A, state=p), p
    return [("rms_norm", lambda: ssd.rms_norm(x, w, r)), ("rms_norm int8", lambda: ssd.rms_norm(x, w, r, format="int8")),
            ("rms_norm_backward", lambda: ssd.rms_norm_backward(x, r, w)),
            ("linear", lambda: (ssd.linear(x, W, activation="silu"),)),
            ("linear_backward", lambda: ssd.linear_backward(dy, x, W, pre=dy, activation="gelu", with_bias=True)),
            ("gated_recurrence", lambda: ssd.gated_recurrence(x, r, A)),
            ("gated_recurrence_backward", lambda: ssd.gated_recurrence_backward(x, x, r, A, saved=saved)),
            ("gated_recurrence_step", step)]


def flat(v):
    return [t for t in (v if isinstance(v, tuple) else (v,)) if t is not None]


@pytest.mark.parametrize("k", range(8))
def test_another_stream_and_graphs(k):
    """A call runs on the current stream, and captured into a graph it gives the eager call's bits at every replay, with
    eager work between the replays."""
    name, call = some_calls(gen(71))[k]
    say("streams and graphs", name)
    want = [t.clone() for t in flat(call())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = flat(call())
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = flat(call())
    for _ in range(3):
        for t in kept:
            t.view(torch.uint8).fill_(0x5a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, kept)), name
        again = flat(call())
        assert all(torch.equal(a, b) for a, b in zip(want, again))


def test_two_calls_at_once_with_workspaces_of_their_own():
    g = gen(72)
    x, gate, A = rn(g, 1, 3000, 64).cuda(), rn(g, 1, 3000, 64).cuda(), -torch.ones(64).cuda()
    want = ssd.gated_recurrence(x, gate, A)
    other = ssd.gated_recurrence(gate, x, A)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(a):
            p = ssd.gated_recurrence(x, gate, A)
        with torch.cuda.stream(b):
            q = ssd.gated_recurrence(gate, x, A)
        torch.cuda.synchronize()
        assert torch.equal(p[0], want[0]) and torch.equal(q[0], other[0])
