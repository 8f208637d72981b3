"""The 64-bit loops of selective_ref.py against differences, and against a known case; CPU only."""
import torch

import selective_ref as ref


def rnd(g, *s):
    return torch.randn(*s, generator=g, dtype=torch.float64)


def test_scan_gradients_are_the_loops_differences():
    g = torch.Generator().manual_seed(1)
    B, L, D, N, G, S = 2, 6, 4, 3, 2, 4
    seq = torch.tensor([[0, 0, 2, 2, 2, -1], [3, 3, 3, 3, 1, 1]], dtype=torch.int32)
    rr = ref.runs(B, L, seq)
    p = [rnd(g, B, L, D), rnd(g, B, L, D), -rnd(g, D, N).abs(), rnd(g, B, L, G, N), rnd(g, B, L, G, N), rnd(g, D), rnd(g, D),
         rnd(g, B, L, D), rnd(g, S, D, N)]
    w, v = rnd(g, B, L, D), rnd(g, S, D, N)
    got = ref.scan_grads(w, v, *p, S, True, rr)

    def value(q):
        out, fin, _, _ = ref.scan(*q, S, True, rr)
        return float((out * w).sum() + (fin * v).sum())
    for i, k in enumerate(("dx", "ddt", "dA", "dB", "dC", "dD", "dbias", "dz", "dh0")):
        d = rnd(g, *p[i].shape)
        hi, lo = list(p), list(p)
        hi[i], lo[i] = p[i] + 1e-6 * d, p[i] - 1e-6 * d
        slope = (value(hi) - value(lo)) / 2e-6
        assert abs(slope - float((got[k] * d).sum())) <= 1e-7 * (1 + abs(slope)), k


def test_conv_gradients_are_the_loops_differences():
    g = torch.Generator().manual_seed(2)
    B, L, Ch, W, S = 2, 7, 3, 4, 5
    seq = torch.tensor([[0, 2, 2, 2, 2, 2, -1], [4, 4, 1, 1, 1, 1, 1]], dtype=torch.int32)
    rr = ref.runs(B, L, seq)
    p = [rnd(g, B, L, Ch), rnd(g, Ch, W), rnd(g, Ch), rnd(g, S, Ch, W - 1)]
    w, v = rnd(g, B, L, Ch), rnd(g, S, Ch, W - 1)
    got = ref.conv_grads(w, v, *p, S, "silu", rr)

    def value(q):
        _, out, fin = ref.conv(*q, S, "silu", rr)
        return float((out * w).sum() + (fin * v).sum())
    for i in range(4):
        d = rnd(g, *p[i].shape)
        hi, lo = list(p), list(p)
        hi[i], lo[i] = p[i] + 1e-6 * d, p[i] - 1e-6 * d
        slope = (value(hi) - value(lo)) / 2e-6
        assert abs(slope - float((got[i] * d).sum())) <= 1e-7 * (1 + abs(slope)), i


def test_scan_with_one_decay_is_a_geometric_sum():
    """Constant inputs: h after t tokens is the geometric sum of the decays."""
    L, d, a, b = 10, 0.5, -0.3, 2.0
    one = torch.ones(1, L, 1, dtype=torch.float64)
    A = torch.full((1, 8), a, dtype=torch.float64)
    B = torch.full((1, L, 1, 8), b, dtype=torch.float64)
    y, fin, _, _ = ref.scan(one, d * one, A, B, B, None, None, None, None, 1, False, ref.runs(1, L))
    r = torch.exp(torch.tensor(d * a, dtype=torch.float64))
    want = d * b * (1 - r ** L) / (1 - r)
    assert torch.allclose(fin, want.expand(1, 1, 8), rtol=1e-13) and torch.allclose(y[0, -1, 0], 8 * b * want, rtol=1e-13)


def test_cache_values_of_e_four_m_three():
    """The reference's codes times scale 1 are the values of the type."""
    vals = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    v = torch.cat([vals, torch.tensor([448.0])]).view(1, 128)
    back, scale = ref.cache(v, 128, "e4m3")
    assert scale.item() == 1.0 and torch.equal(back.float(), v)
