"""dg of heads that forget fast, slowly and wholly, each by its own norm, against the 64-bit
definition."""
import pytest
import torch

import delta_ref as ref
from gpu_common import need_gpu, say
from linear_ref import lengths
from test_gpu_delta import ARGS, BF, F32, _rand, make

pytestmark = pytest.mark.gpu

# A value is its window's anchor, <S, Y> over the state's elements, and up to 256 tokens' summands
# of two parts each.  A part is off by some 8 roundings of 2^-24, at random: its weights' exponents (x of
# them rounds by |x| 2^-24, here up to 30), three fp32 products, an operand's three terms, its sums
# over channels and columns.  512 such errors at random make sqrt(512) 8 2^-24 = 1.1e-5 of a summand,
# which is of a head's typical dg; the anchor's, which all tokens of a window share and which is larger
# where dS_T is, is 2^-24 of the state's norms times the square root of 256 tokens: 16 2^-24 = 1e-6 times
# what it exceeds a typical dg by (here up to 10).  Parts that cancel lose more: 2e-5 to
# 2e-4 at g = -3, 5e-3 to 3e-2 at -10, many times the norm at -20.
LIMIT = 1.1e-5
RATES = (0.01, 0.3, 3.0, 5.0, 10.0, 20.0)


def head_errors(got, want, lens):
    """|got - want| / |want| of each head of each sequence that has tokens"""
    err = (got.double().cpu() - want).norm(dim=1) / want.norm(dim=1)
    return err[torch.tensor([n > 0 for n in lens])]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,Hk,dk,dv,lens,state", [
    (2, 100, 6, 64, 64, None, True), (1, 600, 3, 128, 128, None, False), (4, 290, 2, 32, 64, [290, 257, 1, 64], True),
    (1, 1100, 6, 128, 32, None, True)])
def test_each_head_by_its_own_norm(B, T, Hk, dk, dv, lens, state, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("dg by heads", B, T, Hk, dk, dv, lens, state, dtype)
    H = len(RATES)
    x, gen = make(B, T, H, Hk, dk, dv, dtype, seed=T, state=state, lens=lens)
    x["g"] = -torch.tensor(RATES, device="cuda") * (1.0 + 0.1 * _rand(gen, B, T, H)).clamp(0.5, 1.5)
    dO = _rand(gen, *x["v"].shape).to(dtype)
    dS_T = _rand(gen, B, H, dk, dv) if state else None
    got = kda.delta_backward(*(x[n] for n in ARGS[:5]), dO, x["scale"], x["S0"], dS_T, x["lens"])["dg"]
    torch.cuda.synchronize()
    want = ref.backward(*(x[n] for n in ARGS), dO, x["S0"], dS_T, x["lens"])[0]["dg"]
    n = lengths(x["lens"], B, T)
    for b in range(B):
        if n[b] == 1 and not state:
            n[b] = 0                                # without a state before or behind it a token has no dg
    err = head_errors(got, want, n)
    say([f"{e:.1e}" for e in err.amax(0).tolist()])
    assert (err < LIMIT).all(), err


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decays_of_zero(dtype):
    """Where a token forgets all (exp(g) is 0 in fp32) dg is exactly zero, and what lies before it has
    nothing of what lies behind."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    B, T, H, d = 2, 700, 4, 64
    x, gen = make(B, T, H, H, d, d, dtype, seed=3)
    x["g"] = -0.05 * _rand(gen, B, T, H).abs()
    x["g"][:, :, 0] = float("-inf")
    x["g"][:, 5::37, 1] = -1e30
    x["g"][:, 300, 2] = -104.0
    x["g"][:, 699, 2] = float("-inf")
    x["g"][:, ::64, 3] = -20000.0
    dO, dS_T = _rand(gen, *x["v"].shape).to(dtype), _rand(gen, B, H, d, d)
    got = kda.delta_backward(*(x[n] for n in ARGS[:5]), dO, x["scale"], x["S0"], dS_T)["dg"]
    torch.cuda.synchronize()
    assert (got[x["g"] <= -104.0] == 0).all()
    want = ref.backward(*(x[n] for n in ARGS), dO, x["S0"], dS_T)[0]["dg"]
    err = head_errors(got[..., 1:], want[..., 1:], [T] * B)
    say([f"{e:.1e}" for e in err.amax(0).tolist()])
    assert (err < LIMIT).all(), err
