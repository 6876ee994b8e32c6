"""The kernels that large calls of linear attention run, against the 64-bit sums over pairs: two
column tiles a wave (d = 128 columns in 96 or more sequences x heads x passes), one bf16 term of
the state and the pair weights (bf16 segments of more than 128 tokens; bf16 trees of 512 or more
sequences x heads), and several segments of each."""
import pytest
import torch

import linear_pairs as pairs
import linear_ref as ref
from gpu_common import need_gpu, say
from test_gpu_linear import BF, F32, _rand, _tree, absolute, make, terms

pytestmark = pytest.mark.gpu


def compare(got, form, x, names, args, dtype, exact, n):
    """bf16: one rounding on each part of a sum, but none in states (`exact`: fp32 throughout)."""
    a = absolute(x)
    want, mag = form(*(x[i] for i in args)), form(*(a[i] for i in args))
    if not isinstance(want, dict):
        want, mag = dict(zip(names, want)), dict(zip(names, mag))
    for name in names:
        ref.check(name, got[name], want[name], mag[name], dtype, 1 if dtype == BF and name not in exact else 0, n)


FWD = ("q", "k", "v", "g", "scale", "S0", "lens")
BWD = ("q", "k", "v", "g", "scale", "dO", "S0", "dS_T", "lens")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size,lens,state", [  # B, T, H, Hk, dk, dv
    ((3, 33, 32, 32, 128, 128), None, False),                   # two tiles a wave
    ((3, 161, 32, 8, 32, 128), [161, 97, 0], True),
    ((3, 161, 32, 32, 64, 128), None, True),
    ((3, 161, 32, 16, 128, 128), [1, 161, 130], True),
    ((3, 1100, 32, 8, 128, 128), None, True),                   # and two segments (fp32 five)
    ((3, 1100, 32, 32, 128, 128), [1100, 385, 800], True),
    ((2, 300, 32, 32, 128, 128), None, False),                  # one tile, one term, one segment
    ((2, 1100, 16, 4, 128, 128), None, True),                   # several segments
    ((1, 2500, 8, 8, 128, 128), None, True)])
def test_prefill(size, lens, state, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("prefill", size, lens, state, dtype)
    B, T, H, Hk, dk, dv = size
    x, _ = make(*size, dtype, seed=T + dk, state=state, lens=lens)
    o, S_T = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["scale"], x["S0"], x["lens"])
    torch.cuda.synchronize()
    compare(dict(o=o, S_T=S_T), pairs.prefill, x, ("o", "S_T"), FWD, dtype, ("S_T",), terms(2 * T, dk))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size,lens,state", [
    ((1, 161, 32, 32, 128, 128), None, True),                   # two tiles a wave, the passes in one launch
    ((1, 1100, 32, 8, 128, 128), None, True),                   # and five segments
    ((2, 700, 16, 16, 128, 128), [700, 433], False),
    ((3, 161, 32, 8, 64, 128), None, True),                     # dv with two tiles, dq and dk with one
    ((3, 300, 32, 32, 128, 64), [300, 0, 201], True),           # dq and dk with two
    ((2, 161, 32, 4, 128, 32), None, False),
    ((1, 1500, 8, 8, 128, 128), None, True),                    # one tile, eight segments
    ((2, 600, 8, 4, 32, 128), None, True)])
def test_backward(size, lens, state, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("backward", size, lens, state, dtype)
    B, T, H, Hk, dk, dv = size
    x, gen = make(*size, dtype, seed=T + dv, state=state, lens=lens)
    x["dO"] = _rand(gen, *x["v"].shape).to(dtype)
    x["dS_T"] = _rand(gen, B, H, dk, dv) if state else None
    got = kda.linear_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], x["scale"], x["S0"], x["dS_T"], x["lens"])
    torch.cuda.synchronize()
    compare(got, pairs.backward, x, ("dq", "dk", "dv", "dS0"), BWD, dtype, ("dS0",),
            terms(2 * T, max(dk, dv), H // Hk))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [(16, 13, 32, 8, 128, 128), (16, 64, 32, 32, 128, 128), (16, 47, 32, 32, 64, 128),
                                  (16, 33, 32, 16, 128, 64), (16, 64, 32, 8, 32, 32)])
def test_tree(size, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("tree", size, dtype)
    B, T, H, Hk, dk, dv = size
    assert B * H >= 512
    x, gen = make(*size, dtype, seed=T)
    parent = _tree(gen, B, T)
    o = kda.linear_tree(x["q"], x["k"], x["v"], x["g"], x["S0"], parent, x["scale"])
    torch.cuda.synchronize()
    x["parent"] = parent
    a = absolute({n: t for n, t in x.items() if n != "parent"})
    args = ("q", "k", "v", "g", "scale", "S0")
    ref.check("o", o, pairs.tree(*(x[n] for n in args), parent), pairs.tree(*(a[n] for n in args), parent), dtype,
              1 if dtype == BF else 0, terms(T, dk))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("Hk", [4, 1])
def test_padded_gradients_in_several_segments(Hk, dv, dtype):
    """Sequences that end in the first, a middle and the last of four or more segments, one of no
    tokens and one of a single one; their padding holds NaN and is neither read nor written."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    lens = [700, 0, 1, 97, 256, 333]
    B, T, H, dk = len(lens), 700, 4, 64
    say("padded segments", Hk, dv, dtype)
    assert kda.kda_linear_backward_workspace_bytes(B, T, H, H, dk, dv, dtype) > 0      # segments' states
    x, gen = make(B, T, H, Hk, dk, dv, dtype, seed=Hk + dv, lens=lens)
    x["dO"], x["dS_T"] = _rand(gen, *x["v"].shape).to(dtype), _rand(gen, B, H, dk, dv)
    for b, n in enumerate(lens):
        for t in ("q", "k", "v", "dO"):
            x[t][b, n:] = float("nan")
    out = {n: torch.full_like(x[n[1:]], 7.0) for n in ("dq", "dk", "dv")}
    got = kda.linear_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], x["scale"], x["S0"], x["dS_T"], x["lens"], **out)
    o = torch.full_like(x["v"], 7.0)
    _, S_T = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["scale"], x["S0"], x["lens"], o=o)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        for t in (*out.values(), o):
            assert (t[b, n:] == 7.0).all()
            t[b, n:] = 0
    assert torch.equal(got["dS0"][1], x["dS_T"][1]) and torch.equal(S_T[1], x["S0"][1])
    n = terms(2 * T, dv, H // Hk)
    compare(got, pairs.backward, x, ("dq", "dk", "dv", "dS0"), BWD, dtype, ("dS0",), n)
    compare(dict(o=o, S_T=S_T), pairs.prefill, x, ("o", "S_T"), FWD, dtype, ("S_T",), n)
