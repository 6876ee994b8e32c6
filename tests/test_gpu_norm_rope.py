"""The norm of queries and keys with the position rotation on the GPU against
its 64-bit definition, forward and gradients."""
import pytest
import torch

import linear_ref as ref
from gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(B, T, H, Hk, d, rot, dtype, weights, far=0, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = dict(q=(2.0 * r(B, T, H, d)).to(dtype), k=(0.5 * r(B, T, Hk, d)).to(dtype),
             dy_q=r(B, T, H, d).to(dtype), dy_k=r(B, T, Hk, d).to(dtype),
             w_q=1 + r(d) if weights else None, w_k=1 + r(d) if weights else None,
             inv_freq=10000.0 ** (-torch.arange(0, rot, 2, device="cuda") / rot) if rot else None,
             positions=(torch.arange(T, device="cuda").expand(B, T) + far).to(torch.int32) if rot else None)
    return x


# The rotation's cos and sin come from an angle in fp32 within [-pi, pi] (off by at
# most pi 2^-24) and are good to a few 2^-24: 16 in units of 2^-24; the norm's sum
# of d squares adds d.
def terms(d, rows=0):
    return d + rows + 32


def check(x, got, names, norm, eps, il):
    dt, d = x["q"].dtype, x["q"].shape[-1]
    for name, y in zip(names, got):
        n = name[-1]
        want, mag = ref.norm_rope(x[n], x["w_" + n], x["positions"], x["inv_freq"], norm, eps, il)
        ref.check(name, y, want, mag, dt, 0, terms(d))


CASES = [  # B, T, H, Hk, d, rot, weights
    (1, 1, 1, 1, 32, 32, True), (2, 3, 4, 1, 64, 2, False), (1, 17, 5, 3, 128, 128, True),
    (2, 9, 8, 8, 128, 64, False), (1, 33, 3, 2, 64, 38, True), (2, 5, 2, 2, 32, 0, True), (1, 130, 33, 7, 128, 126, True),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm,il", [("l2", False), ("rms", True), ("l2", True), ("rms", False)])
@pytest.mark.parametrize("case", CASES)
def test_forward_and_gradients(case, norm, il, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("norm rope", case, norm, il, dtype)
    B, T, H, Hk, d, rot, weights = case
    x = make(B, T, H, Hk, d, rot, dtype, weights, seed=T)
    kw = dict(w_q=x["w_q"], w_k=x["w_k"], norm=norm, eps=1e-5, interleaved=il)
    y = kda.qk_norm_rope(x["q"], x["k"], x["positions"], x["inv_freq"], **kw)
    got = kda.qk_norm_rope_backward(x["q"], x["k"], x["positions"], x["inv_freq"], x["dy_q"], x["dy_k"], **kw)
    torch.cuda.synchronize()
    check(x, y, ("y_q", "y_k"), norm, 1e-5, il)
    for n in "qk":
        dx, mx, dw, mw = ref.norm_rope_backward(x[n], x["w_" + n], x["positions"], x["inv_freq"], x["dy_" + n],
                                                norm, 1e-5, il)
        ref.check("d" + n, got["d" + n], dx, mx, dtype, 0, 2 * terms(d))
        if weights:
            rows = B * T * x[n].shape[2]
            ref.check("dw_" + n, got["dw_" + n], dw, mw, dtype, 0, terms(d, rows))
        else:
            assert got["dw_" + n] is None


@pytest.mark.parametrize("far", [10 ** 6, 2 ** 31 - 40, -(2 ** 31)])
def test_far_positions(far):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x = make(1, 20, 2, 2, 64, 64, F32, False, far=far)
    y = kda.qk_norm_rope(x["q"], x["k"], x["positions"], x["inv_freq"], norm="l2")
    torch.cuda.synchronize()
    check(x, y, ("y_q", "y_k"), "l2", 1e-6, False)


def test_zero_rows_in_place_and_no_rotation():
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x = make(2, 6, 3, 1, 128, 64, BF, True)
    x["q"][0, 1] = 0
    y = kda.qk_norm_rope(x["q"], x["k"], x["positions"], x["inv_freq"], w_q=x["w_q"], w_k=x["w_k"])
    assert (y[0][0, 1] == 0).all()
    g = kda.qk_norm_rope_backward(x["q"], x["k"], x["positions"], x["inv_freq"], x["dy_q"], x["dy_k"],
                                  w_q=x["w_q"], w_k=x["w_k"])
    assert all(torch.isfinite(t.float()).all() for t in g.values())
    # in place: y over x, dx over dy
    q, k = x["q"].clone(), x["k"].clone()
    kda.kda_qk_norm_rope(q, k, x["w_q"], x["w_k"], x["positions"], x["inv_freq"], "rms", 1e-6, False, q, k)
    assert torch.equal(q, y[0]) and torch.equal(k, y[1])
    dq, dk = x["dy_q"].clone(), x["dy_k"].clone()
    kda.kda_qk_norm_rope_backward(x["q"], x["k"], x["w_q"], x["w_k"], x["positions"], x["inv_freq"], "rms", 1e-6,
                                  False, dq, dk, dq, dk, None, None)
    assert torch.equal(dq, g["dq"]) and torch.equal(dk, g["dk"])


def test_captured_calls_replay():
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x = make(2, 70, 6, 2, 128, 128, BF, True)

    def work():
        y = kda.qk_norm_rope(x["q"], x["k"], x["positions"], x["inv_freq"], w_q=x["w_q"], w_k=x["w_k"])
        g = kda.qk_norm_rope_backward(x["q"], x["k"], x["positions"], x["inv_freq"], x["dy_q"], x["dy_k"],
                                      w_q=x["w_q"], w_k=x["w_k"])
        return [*y, *g.values()]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for _ in range(3):
        x["q"].mul_(0.5)
        x["dy_k"].add_(0.25)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, work()):
            assert torch.equal(a, b)


def test_gradients_of_zero_rows_under_the_smallest_eps():
    """eps 2^-133 (exact in fp32): r is 2^66.5 on a row of zeros, its square past fp32."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x = make(1, 5, 2, 2, 64, 64, F32, True)
    x["q"][0, 1:3] = 0
    eps = 2.0 ** -133
    got = kda.qk_norm_rope_backward(x["q"], x["k"], x["positions"], x["inv_freq"], x["dy_q"], x["dy_k"],
                                    w_q=x["w_q"], w_k=x["w_k"], eps=eps)
    torch.cuda.synchronize()
    for n in "qk":
        dx, mx, dw, mw = ref.norm_rope_backward(x[n], x["w_" + n], x["positions"], x["inv_freq"], x["dy_" + n],
                                                "rms", eps, False)
        ref.check("d" + n, got["d" + n], dx, mx, F32, 0, 2 * terms(64))
        ref.check("dw_" + n, got["dw_" + n], dw, mw, F32, 0, terms(64, 10))
