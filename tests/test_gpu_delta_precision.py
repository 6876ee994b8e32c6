"""The error in norm of each head's results of the gated delta rule against 64 bits, with limits
that tell an operand in two bf16 terms from one in three, and one term from two in bf16's o."""
import pytest
import torch

import delta_ref as ref
from delta_precision import errors, inputs, limit
from gpu_common import need_gpu, say
from test_gpu_delta import ARGS, BF, F32

pytestmark = pytest.mark.gpu

HEADS = dict(o=2, S_T=1, dq=2, dk=2, dv=2, dbeta=2, dS0=1)


def run(x):
    import linear_attention_recurrence_05_amd as kda
    y = {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in x.items()}
    o, S_T = kda.delta_prefill(*(y[n] for n in ARGS), y["S0"])
    got = kda.delta_backward(*(y[n] for n in ARGS[:5]), y["dO"], y["scale"], y["S0"], y["dS_T"])
    torch.cuda.synchronize()
    return {**got, "o": o, "S_T": S_T}


def check(x, names=tuple(HEADS)):
    got = run(x)
    out = ref.prefill(*(x[n] for n in ARGS), x["S0"])
    want = {"o": out["o"], "S_T": out["S_T"]}
    if set(names) - set(want):
        want.update(ref.backward(*(x[n] for n in ARGS), x["dO"], x["S0"], x["dS_T"])[0])
    err = {n: errors(got[n], want[n], HEADS[n]) for n in names}
    say({n: f"{e:.1e}" for n, e in err.items()})
    for n, e in err.items():
        assert e < limit(n, x["q"].dtype), (n, e)


# The last three have three and more of dg's anchors.
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [  # B, T, H, Hk, dk, dv
    (1, 16, 8, 8, 32, 32), (1, 300, 4, 4, 64, 64), (2, 161, 3, 3, 128, 32), (1, 200, 4, 2, 32, 128), (1, 900, 2, 1, 128, 128),
    (1, 1300, 2, 2, 64, 32), (2, 700, 3, 3, 32, 64)])
def test_prefill_and_gradients(size, dtype):
    need_gpu()
    say("precision", size, dtype)
    check(inputs(*size, dtype, seed=size[1]))


@pytest.mark.parametrize("size", [(1, 300, 4, 4, 64, 64), (1, 256, 4, 2, 128, 128), (2, 90, 4, 4, 32, 32)])
def test_gradients_where_queries_and_keys_are_alike(size):
    need_gpu()
    say("precision, alike", size)
    check(inputs(*size, BF, seed=size[1], queries=True))


@pytest.mark.parametrize("dk", [32, 64, 128])
def test_many_heads(dk):
    """A workgroup for each head (from 128 of them and 128 value columns on)."""
    need_gpu()
    say("precision, many heads", dk)
    check(inputs(4, 130, 32, 16, dk, 128, BF, seed=dk, queries=True), ("o", "S_T"))


@pytest.mark.parametrize("size", [(1, 1, 1, 1, 128, 128), (1, 1, 32, 32, 128, 128), (2, 3, 4, 2, 64, 64), (1, 64, 8, 8, 32, 32),
                                  (1, 300, 4, 4, 64, 64), (1, 256, 4, 4, 128, 128), (1, 333, 4, 1, 32, 128)])
def test_bf16_outputs_have_their_own_rounding_alone(size):
    """Also of prompts of a token and of a chunk without a state, and where queries and keys have most
    of their length in common."""
    need_gpu()
    say("precision of o", size)
    for queries in (False, True):
        x = inputs(*size, BF, seed=size[1], queries=queries)
        x["S0"].zero_()
        check(x, ("o", "S_T"))
