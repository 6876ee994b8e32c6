"""The ring plan on streams of several hardware queues: the XCD that a launch's
first workgroup runs on differs from queue to queue (and changes for a queue
as others come into use), and a unit's workgroups have to share one XCD, whichever it is."""
import pytest
import torch

import linear_attention_recurrence_05_amd as kda
from gpu_common import need_gpu, plan, say
from linear_attention_recurrence_05_amd.inputs import prefill_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,H", [(2, 100, 3), (1, 1000, 32)])
def test_ring_plan_on_many_streams(B, T, H):
    """Bit for bit the split plan's results on every stream, and on the default one after each."""
    dev = need_gpu()
    x = prefill_inputs(B, T, H, 128, 128, torch.bfloat16, seed=B * 1000 + T, s0_std=0.1, device=dev)
    args = [x[n] for n in ("q", "k", "v", "z", "beta", "A", "g_min", "S0")]
    assert kda.kda_chunk_prefill_plan(B, T, H, 128, 128, torch.bfloat16) == "ring"
    with plan("split"):
        o, S = kda.chunk_prefill(*args)
    torch.cuda.synchronize()
    for i in range(9):
        stream = torch.cuda.Stream()
        for s in (stream, torch.cuda.default_stream()):
            with torch.cuda.stream(s):
                got = kda.chunk_prefill(*args)
            s.synchronize()
            say("stream", i, "default" if s is not stream else "", torch.equal(got[0], o), torch.equal(got[1], S))
            assert torch.equal(got[0], o) and torch.equal(got[1], S)
