"""Gradients of a long sequence a part at a time: each part's states and their gradients handed on."""
import pytest
import torch

import delta_ref as ref
from delta_precision import errors, limit
from gpu_common import need_gpu, say
from test_gpu_delta import ARGS, BF, F32, _rand, make
from test_gpu_delta_gates import LIMIT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cuts", [(0, 400, 500), (0, 64, 65, 320, 500)])
def test_parts_of_a_sequence(cuts, dtype):
    """Within the limits of a whole call, every part."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("gradients in parts", cuts, dtype)
    x, gen = make(2, 500, 4, 2, 64, 64, dtype, seed=2)
    dO, dS = _rand(gen, *x["v"].shape).to(dtype), _rand(gen, *x["S0"].shape)
    want = ref.backward(*(x[n] for n in ARGS), dO, x["S0"], dS)[0]
    parts = [[x[n][:, a:b].contiguous() for n in ARGS[:5]] + [dO[:, a:b].contiguous()] for a, b in zip(cuts, cuts[1:])]
    states = [x["S0"]]
    for p in parts[:-1]:
        states.append(kda.delta_prefill(*p[:5], x["scale"], states[-1])[1])
    out, dS_T = [], dS
    for p, S0 in zip(reversed(parts), reversed(states)):
        out.append(kda.delta_backward(*p, x["scale"], S0, dS_T))
        dS_T = out[-1]["dS0"]
    torch.cuda.synchronize()
    for n in ("dq", "dk", "dv", "dbeta", "dg"):
        got = torch.cat([o[n] for o in reversed(out)], 1)
        assert errors(got, want[n], 2) < (LIMIT if n == "dg" else limit(n, dtype)), n
    assert errors(dS_T, want["dS0"], 1) < limit("dS0", dtype)
