"""GPU tests of every tile of the matrix product, at the sizes of linear_tiles.py, all outputs against products in 64 bits
(on the device, from the definitions).  Tolerances are those of test_gpu_layer.py: two roundings a product, 20 behind the
sum, 60 for an activation, half a step for dpre's rounding, half a step of the output's type.  e4m3 goes to outputs of 32
bits and of 16, whose instruction cuts seven of eight products at 2^-13 of the largest at most: 7 * 2^11 u more."""
import pytest
import torch

import layer_ref as ref
import mamba_ssd_prefill_amd as ssd
from gpu_common import require_gpu, say
from linear_tiles import GRADIENTS, PRODUCTS

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def dev():
    return require_gpu()


def close(got, want, scale, roundings, name):
    """layer_ref.close on the device: |got - want| <= eps / 2 |want| + roundings u scale (plus the type's smallest steps)."""
    fi = torch.finfo(got.dtype)
    tol = (1 + fi.eps) * (fi.eps / 2 * want.abs() + roundings * ref.U * scale) + fi.smallest_normal * fi.eps
    bad = ~((got.double() - want).abs() <= tol)
    if bad.any():
        at = bad.nonzero()
        raise AssertionError("%s: %d of %d values off, from %s to %s"
                             % (name, len(at), bad.numel(), at[0].tolist(), at[-1].tolist()))


def wide(t):
    return t.float().double()


def operands(M, K, N, dtype, g):
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if dtype in DT:
        return rn(M, K).to(DT[dtype]), (rn(N, K) / K**0.5).to(DT[dtype]), None, None, DT[dtype]
    sx, sw = torch.exp(rn(M)) / 1000, torch.exp(rn(N)) / 100
    if dtype == "int8":
        x, w = (torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8) for s in ((M, K), (N, K)))
    else:
        x, w = ((100 * rn(*s)).clamp(-448, 448).to(torch.float8_e4m3fn) for s in ((M, K), (N, K)))
    return x, w, sx, sw, torch.float32


@pytest.mark.parametrize("case", PRODUCTS, ids=str)
def test_every_tile(case):
    say("tile", case)
    M, K, N, dtype, *_ = case
    g = torch.Generator(device="cuda").manual_seed(81)
    x, w, sx, sw, out = operands(M, K, N, dtype, g)
    for t in (out, torch.float16) if dtype == "e4m3" else (out,):
        check_tile(case, x, w, sx, sw, t, g)


def check_tile(case, x, w, sx, sw, out, g):
    M, K, N, dtype, *_ = case
    b, r = torch.randn(N, generator=g, device="cuda"), torch.randn(M, N, generator=g, device="cuda").to(out)
    args = dict(activation="silu", x_scale=sx, weight_scale=sw, out_dtype=out)
    got, pre = ssd.linear(x, w, b, r, save_pre=True, **args)
    assert torch.equal(ssd.linear(x, w, b, r, **args), got)
    want, S = wide(x) @ wide(w).t(), wide(x).abs() @ wide(w).t().abs()
    for s in () if sx is None else (sx[:, None], sw):
        want, S = want * s.double(), S * s.double()
    want, S = want + b.double(), S + b.double().abs()
    sums = 0 if dtype == "int8" else 2 * K
    if dtype == "e4m3" and out != torch.float32:
        sums += 7 * 2**11
    close(pre, want, S, sums + 20, "pre")
    v = want * torch.sigmoid(want)
    close(got, v + r.double(), 1.2 * S + v.abs() + r.double().abs(), sums + 80, "linear")


@pytest.mark.parametrize("case", GRADIENTS, ids=str)
def test_both_gradients_by_every_tile(case):
    say("gradients' tile", case)
    M, K, N, dtype, _ = case
    g, t = torch.Generator(device="cuda").manual_seed(82), DT[dtype]
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w, dout, pre = rn(M, K).to(t), (rn(N, K) / K**0.5).to(t), rn(M, N).to(t), rn(M, N).to(t)
    got = ssd.linear_backward(dout, x, w, pre=pre, activation="silu", with_bias=True)
    d, S = wide(dout) * ref.dact(wide(pre), "silu"), 1.2 * wide(dout).abs()
    half = torch.finfo(t).eps / 2 / ref.U  # dpre's own rounding
    close(got.dx, d @ wide(w), S @ wide(w).abs(), 2 * N + 80 + half, "dx")
    close(got.dweight, d.t() @ wide(x), S.t() @ wide(x).abs(), 2 * M + 80 + half, "dweight")
    close(got.dbias, d.sum(0), S.sum(0), M + 80, "dbias")
