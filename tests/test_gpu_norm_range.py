"""The norm of queries and keys over the whole range of finite rows and of eps: squares (and
products of gradients with rows) that leave fp32's range, beside ordinary rows in the same call."""
import pytest
import torch

import linear_ref as ref
from gpu_common import need_gpu, say
from test_gpu_norm_rope import BF, F32, check, make, terms

pytestmark = pytest.mark.gpu

# Rows times 2^k and their gradients times 2^j, exact in both types: |x| < 2^125 x 6, and
# every gradient of a row stays within fp32's range (|j - k| <= 100).
ROWS = [(0, 0), (62, 70), (63, 0), (64, 100), (70, 64), (100, 100), (125, 100), (0, 100), (-60, 0), (-75, -90), (125, 30)]


def scaled(x):
    B, T, H, _ = x["q"].shape
    for n in "qk":
        h = x[n].shape[2]
        at = torch.arange(B * T * h, device="cuda").reshape(B, T, h) % len(ROWS)
        for name, col in ((n, 0), ("dy_" + n, 1)):
            s = torch.tensor([2.0 ** r[col] for r in ROWS], device="cuda")[at][..., None]
            x[name] = (x[name].float() * s).to(x[name].dtype)
            assert torch.isfinite(x[name]).all()
    return x


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("eps", [1e-6, 2.0 ** -140, 3e38])
@pytest.mark.parametrize("case", [  # d, rot, interleaved, norm: every way a pair is turned
    (128, 128, False, "l2"), (64, 64, True, "rms"), (32, 0, False, "l2"), (128, 38, False, "rms"), (64, 6, True, "l2")])
def test_any_finite_row(case, eps, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("norm range", case, eps, dtype)
    d, rot, il, norm = case
    eps = float(torch.tensor(eps))                  # as fp32 holds it
    x = scaled(make(2, 7, 5, 3, d, rot, dtype, True, seed=d + rot))
    kw = dict(w_q=x["w_q"], w_k=x["w_k"], norm=norm, eps=eps, interleaved=il)
    y = kda.qk_norm_rope(x["q"], x["k"], x["positions"], x["inv_freq"], **kw)
    got = kda.qk_norm_rope_backward(x["q"], x["k"], x["positions"], x["inv_freq"], x["dy_q"], x["dy_k"], **kw)
    torch.cuda.synchronize()
    check(x, y, ("y_q", "y_k"), norm, eps, il)
    for n in "qk":
        dx, mx, dw, mw = ref.norm_rope_backward(x[n], x["w_" + n], x["positions"], x["inv_freq"], x["dy_" + n],
                                                norm, eps, il)
        ref.check("d" + n, got["d" + n], dx, mx, dtype, 0, 2 * terms(d))
        ref.check("dw_" + n, got["dw_" + n], dw, mw, dtype, 0, terms(d, 14 * x[n].shape[2]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_unit_rows_of_the_largest_values(dtype):
    """A row of one repeated value has 1 / sqrt(d) everywhere, whatever the value."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    big = torch.finfo(BF).max                       # in both types
    q = torch.tensor([1.0, 1e18, 1e19, 2e19, 1e30, big, -big], device="cuda").to(dtype)
    q = q[None, :, None, None].expand(1, 7, 2, 128).contiguous()
    y, _ = kda.qk_norm_rope(q, q, norm="l2", eps=1e-6)
    torch.cuda.synchronize()
    want = torch.sign(q.double()) / 128 ** 0.5
    tol = ref.HALF[dtype] + (terms(128)) * 2.0 ** -24
    assert ((y.double() - want).abs() <= tol * want.abs()).all(), y[0, :, 0, 0]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", [(128, 128, False, "l2"), (64, 64, True, "rms"), (32, 0, False, "l2"),
                                  (128, 38, False, "rms"), (64, 6, True, "l2")])
def test_infinities_and_nan_stay_in_their_rows(case, dtype):
    """Every other row keeps its bits, also beside rows that are taken times a power of two; the
    weights' gradients of the other tensor too."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    d, rot, il, norm = case
    x = make(2, 9, 5, 3, d, rot, dtype, True, seed=d)
    kw = dict(w_q=x["w_q"], w_k=x["w_k"], norm=norm, eps=1e-6, interleaved=il)

    def both():
        y = kda.qk_norm_rope(x["q"], x["k"], x["positions"], x["inv_freq"], **kw)
        g = kda.qk_norm_rope_backward(x["q"], x["k"], x["positions"], x["inv_freq"], x["dy_q"], x["dy_k"], **kw)
        torch.cuda.synchronize()
        return y[0], g["dq"], y[1], g["dk"], g["dw_k"]

    clean = both()
    bad = [(0, 0, 0, "nan"), (0, 3, 2, "inf"), (1, 5, 4, "-inf"), (1, 8, 1, "1e38")]
    for b, t, h, value in bad:
        x["q"][b, t, h, (7 * t + h) % d] = float(value)
    got = both()
    for b, t, h, value in bad[:3]:
        assert not torch.isfinite(got[0][b, t, h].float()).all()
    for b, t, h, value in bad:
        for i in (0, 1):
            got[i][b, t, h] = clean[i][b, t, h]
    for a, c in zip(got, clean):
        assert torch.equal(a, c)
