"""The norm of queries and keys over more tokens than a launch has workgroups (1024 forward, 768
backward), so that each takes several in turn: the next token's rows and angles are fetched while
this one's are used, and the weights' gradients add up over a workgroup's tokens."""
import pytest
import torch

import linear_ref as ref
from gpu_common import need_gpu, say
from test_gpu_norm_rope import BF, F32, check, make, terms

pytestmark = pytest.mark.gpu

B, T, H, HK = 2, 1301, 5, 3      # 2602 tokens: three or four for each workgroup, the last round partly empty


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", [  # d, rot, interleaved, norm: how a lane gets its pairs' other elements
    (128, 0, False, "l2"),         # no rotation
    (128, 128, True, "rms"),       # whole lanes of neighbouring pairs
    (64, 22, True, "l2"),          # a lane turned in part
    (128, 64, False, "l2"),        # halves of whole lanes: from another lane
    (64, 38, False, "rms"),        # any other halves: through LDS
    (32, 32, False, "rms")])
def test_many_tokens(case, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("norm tokens", case, dtype)
    d, rot, il, norm = case
    x = make(B, T, H, HK, d, rot, dtype, True, seed=rot + d)
    if rot:                        # another position at every token of each sequence
        gen = torch.Generator(device="cuda").manual_seed(rot)
        x["positions"] = torch.randint(0, 1 << 20, (B, T), generator=gen, device="cuda").to(torch.int32)
    kw = dict(w_q=x["w_q"], w_k=x["w_k"], norm=norm, eps=1e-5, interleaved=il)
    y = kda.qk_norm_rope(x["q"], x["k"], x["positions"], x["inv_freq"], **kw)
    got = kda.qk_norm_rope_backward(x["q"], x["k"], x["positions"], x["inv_freq"], x["dy_q"], x["dy_k"], **kw)
    # in place: y over x, dx over dy, without the weights' gradients
    q, k, dq, dk = (x[n].clone() for n in ("q", "k", "dy_q", "dy_k"))
    fixed = (x["w_q"], x["w_k"], x["positions"], x["inv_freq"], norm, 1e-5, il)
    kda.kda_qk_norm_rope(q, k, *fixed, q, k)
    kda.kda_qk_norm_rope_backward(x["q"], x["k"], *fixed, dq, dk, dq, dk, None, None)
    torch.cuda.synchronize()
    assert torch.equal(q, y[0]) and torch.equal(k, y[1])
    assert torch.equal(dq, got["dq"]) and torch.equal(dk, got["dk"])
    check(x, y, ("y_q", "y_k"), norm, 1e-5, il)
    for n in "qk":
        dx, mx, dw, mw = ref.norm_rope_backward(x[n], x["w_" + n], x["positions"], x["inv_freq"], x["dy_" + n],
                                                norm, 1e-5, il)
        ref.check("d" + n, got["d" + n], dx, mx, dtype, 0, 2 * terms(d))
        # A lane adds up at most 4 rows of a token for 4 tokens, the workgroup's lanes of
        # an element (at most 64) and then 48 partial sums in 16 parts follow.
        ref.check("dw_" + n, got["dw_" + n], dw, mw, dtype, 0, terms(d, 16 + 64 + 48 + 16))
