"""The error in norm of fp32 results of linear attention, and of states of either type, against 64
bits: small enough that an operand held in two bf16 terms instead of three would show."""
import pytest
import torch

import linear_pairs as pairs
from gpu_common import need_gpu, say
from linear_precision import LIMIT, error, inputs
from test_gpu_linear import BF, F32, _tree

pytestmark = pytest.mark.gpu


def on_gpu(x):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in x.items()}


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("size", [  # B, T, H, Hk, dk, dv
    (1, 300, 8, 8, 64, 64), (2, 500, 4, 4, 32, 128), (1, 600, 8, 4, 128, 128), (1, 400, 4, 2, 128, 64),
    (3, 161, 32, 16, 128, 128), (3, 600, 32, 32, 128, 128), (1, 20, 2, 1, 32, 32)])
def test_prefill_and_gradients(size, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("precision", size, dtype)
    x = on_gpu(inputs(*size, dtype, seed=size[1]))
    args = tuple(x[n] for n in ("q", "k", "v", "g"))
    o, S_T = kda.linear_prefill(*args, x["scale"], x["S0"])
    got = dict(kda.linear_backward(*args, x["dO"], x["scale"], x["S0"], x["dS_T"]), o=o, S_T=S_T)
    torch.cuda.synchronize()
    want = pairs.backward(*args, x["scale"], x["dO"], x["S0"], x["dS_T"])
    want["o"], want["S_T"] = pairs.prefill(*args, x["scale"], x["S0"])
    err = {n: error(got[n], want[n]) for n in want if dtype == F32 or n in ("S_T", "dS0")}
    say({n: f"{e:.1e}" for n, e in err.items()})
    assert max(err.values()) < LIMIT, err


@pytest.mark.parametrize("size", [(2, 64, 4, 2, 64, 128), (16, 64, 32, 8, 128, 128), (3, 17, 2, 2, 32, 32)])
def test_fp32_trees(size):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("precision of a tree", size)
    x = on_gpu(inputs(*size, F32, seed=size[1]))
    parent = _tree(torch.Generator(device="cuda").manual_seed(1), *size[:2])
    args = tuple(x[n] for n in ("q", "k", "v", "g"))
    o = kda.linear_tree(*args, x["S0"], parent, x["scale"])
    torch.cuda.synchronize()
    e = error(o, pairs.tree(*args, x["scale"], x["S0"], parent))
    say(f"{e:.1e}")
    assert e < LIMIT
