"""The gradients of layer_ref.py against autograd through its forward definitions and against differences."""
import pytest
import torch

import layer_ref as ref


def rnd(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed + sum(shape)), dtype=torch.float64)


def differences(f, inputs, grads, step=1e-6):
    """Each gradient against the central difference of the scalar f along one random direction."""
    for k, (v, g) in enumerate(zip(inputs, grads)):
        d = rnd(*v.shape, seed=99 + k)
        up, down = [list(inputs) for _ in range(2)]
        up[k], down[k] = v + step * d, v - step * d
        want = (f(*up) - f(*down)) / (2 * step)
        got = (g * d).sum()
        assert abs(float(got - want)) < 1e-6 * (1 + abs(float(want))), k


def test_norm_gradients():
    s, w, dout, dsum = rnd(5, 7), rnd(7, seed=1), rnd(5, 7, seed=2), rnd(5, 7, seed=3)
    f = lambda s, w: (ref.norm(s, None, w, 1e-3)[1] * dout + s * dsum).sum()  # noqa: E731
    differences(f, (s, w), ref.norm_grads(dout, s, w, dsum, 1e-3))


@pytest.mark.parametrize("kind", [None, "silu", "gelu"])
def test_product_gradients(kind):
    x, w, b, dout = rnd(6, 5), rnd(4, 5, seed=1), rnd(4, seed=2), rnd(6, 4, seed=3)

    def f(x, w, b):
        return (ref.act(x @ w.t() + b, kind) * dout).sum()
    differences(f, (x, w, b), ref.product_grads(dout, x, w, x @ w.t() + b, kind))


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("gated", [True, False])
def test_recurrence_gradients(normalize, gated):
    B, L, D, S = 2, 6, 3, 5
    rr = [(0, 3, 0, 2), (0, 1, 2, 3), (0, -1, 5, 1), (1, 0, 0, 6)]
    x, gate, ig, dout = (rnd(B, L, D, seed=k) for k in range(4))
    A, gb, ib, h0, dfin = -rnd(D, seed=5).abs() - 0.1, rnd(D, seed=6), rnd(D, seed=7), rnd(S, D, seed=8), rnd(S, D, seed=9)
    used = torch.ones(B, L, 1, dtype=torch.float64)
    used[0, 5] = 0

    def f(x, gate, A, ig, gb, ib, h0):
        out, fin, _ = ref.recurrence(x, gate, A, ig if gated else None, gb, ib if gated else None, normalize, h0, S, rr)
        return (out * dout * used).sum() + (fin * dfin).sum()
    got = ref.recurrence_grads(dout, dfin, x, gate, A, ig if gated else None, gb, ib if gated else None, normalize, h0, S, rr)
    if not gated:
        got = got[:3] + (torch.zeros_like(x),) + got[4:5] + (torch.zeros_like(ib),) + got[6:]
    differences(f, (x, gate, A, ig, gb, ib, h0), got)
