"""GPU tests of the gated recurrence under the token-by-token bounds of recurrence_bounds.py, which a state kept or passed between
tiles in fewer than 32 bits does not meet (test_recurrence_bounds.py): decays that forget at once, and ones that keep
a state for hundreds of tokens."""
import pytest
import torch

import layer_ref as ref
import mamba_ssd_prefill_amd as ssd
from gpu_common import require_gpu, say
from recurrence_bounds import Bounds
from test_gpu_layer import DT, REC, rec_case, rn, used

pytestmark = pytest.mark.gpu
NAMES = ("dx", "dgate", "dA", "din_gate", "dgate_bias", "din_bias", "dh0")


@pytest.fixture(scope="module", autouse=True)
def dev():
    return require_gpu()


def check(case, slow):
    say("recurrence, bounds by token", case, slow)
    B, L, D, dtype, st, *_ = case
    ins, h0, seq, S, args, kw, g = rec_case(case, 91)
    if slow:
        A = torch.log(0.9 + 0.099 * torch.rand(D, generator=g))
        ins, args[2] = ins[:2] + (A,) + ins[3:], A.cuda()
    dout, dfin = rn(g, B, L, D).to(ins[0].dtype), rn(g, S, D).to(DT[st])
    out, fin, saved = ssd.gated_recurrence(*args, **kw, save_for_backward=True)
    got = ssd.gated_recurrence_backward(dout.cuda(), *args, saved=saved, dfinal_state=dfin.cuda(), **kw)
    torch.cuda.synchronize()
    rr, norm, dout = ref.runs(B, L, seq), case[9], used(dout, seq, S)
    bound = Bounds(*ins, norm, h0, S, rr, dout, dfin)
    want, wfin, _ = ref.recurrence(*ins, norm, h0, S, rr)
    ref.close(out, want, bound.out, 1, ins[0].dtype, "out")
    ref.close(fin, wfin, bound.fin, 1, DT[st], "final state")
    grads = ref.recurrence_grads(dout, dfin, *ins, norm, h0, S, rr)
    for v, w, e, name in zip(got, grads, bound.grads, NAMES):
        if v is not None:
            ref.close(v, w, e, 1, v.dtype, name)


@pytest.mark.parametrize("slow", [False, True])
@pytest.mark.parametrize("case", REC, ids=str)
def test_recurrence_token_by_token(case, slow):
    check(case, slow)


@pytest.mark.parametrize("dtype,gated", [("f32", True), ("f16", False)])
def test_recurrence_across_many_tiles(dtype, gated):
    """70 tiles forward and 140 backward, states that last: those passed between tiles decide the outputs behind them."""
    check((1, 8900, 40, dtype, "f32", None, True, gated, True, True, False), True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,extra,shift", [(66, 1, 1), (64, 3, 0), (66, 2, 1), (65, 1, 1)])
def test_recurrence_rows_that_start_anywhere(D, extra, shift, dtype):
    """Rows on their elements' alignment alone: the bits of aligned ones, forward, backward and for one token."""
    say("rows that start anywhere", D, extra, shift, dtype)
    B, L, g = 2, 200, torch.Generator().manual_seed(92)
    whole = [rn(g, B, L, D).to(DT[dtype]).cuda() for _ in range(3)]

    def moved(t):
        flat = torch.full((t[..., 0].numel() * (D + extra) + 8,), float("nan"), dtype=t.dtype, device="cuda")
        lead = t.shape[:-1]
        rows = flat[shift:shift + t[..., 0].numel() * (D + extra)].view(*lead, D + extra)[..., :D]
        rows.copy_(t)
        return rows
    A, dout = -torch.exp(rn(g, D) - 2).cuda(), rn(g, B, L, D).to(DT[dtype]).cuda()
    results = []
    for x, gate, ig in (whole, [moved(t) for t in whole]):
        out, fin, saved = ssd.gated_recurrence(x, gate, A, ig, save_for_backward=True)
        grads = ssd.gated_recurrence_backward(dout, x, gate, A, ig, saved=saved)
        pool = fin.clone()
        one = ssd.gated_recurrence_step(x[:, 3], gate[:, 3], A, ig[:, 3], state=pool)
        results.append([out, fin, one, pool] + [v for v in grads if v is not None])
    assert all(torch.equal(a, b) for a, b in zip(*results))
