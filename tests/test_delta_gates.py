"""The form in which the gradients' kernels sum up dg keeps its digits for heads that forget fast
(CPU model of that sum of fp32 parts, against the definition in 64 bits)."""
import pytest
import torch

import delta_ref as ref


def sums(x, dO, dS_T, dtype, kept):
    """dg as a sum from each token to the sequence's end.  kept: each token's summand is of what
    older and later tokens leave alone, so that it has the factor of a decay; else it is dO . o -
    dv . v, whose parts cancel where a token forgets all."""
    f = lambda t: t.to(dtype)  # noqa: E731
    q, k, v, beta, dO, Y = f(x["q"]), f(x["k"]), f(x["v"]), f(x["beta"]), f(dO), f(dS_T)
    a, scale, (B, T, H, _) = torch.exp(f(x["g"])), x["scale"], v.shape
    S, old, kS, dots = f(x["S0"]), [], [], torch.zeros(B, T, H, dtype=dtype)
    for t in range(T):
        S = a[:, t, :, None, None] * S
        kS.append((k[:, t, :, :, None] * S).sum(2))
        old.append(scale * (q[:, t, :, :, None] * S).sum(2))
        end = S - k[:, t, :, :, None] * (beta[:, t, :, None] * kS[t])[:, :, None]   # S_t less what v wrote
        S = end + k[:, t, :, :, None] * (beta[:, t, :, None] * v[:, t])[:, :, None]
    total = ((end if kept else S).double() * Y.double()).sum((2, 3))
    for t in reversed(range(T)):
        p = scale * (q[:, t] * k[:, t]).sum(-1)[..., None]
        b = beta[:, t, :, None]
        yK = (k[:, t, :, :, None] * Y).sum(2)
        dv = b * (yK + p * dO[:, t])
        if kept:
            dots[:, t] = (dO[:, t] * (old[t] - b * p * kS[t])).sum(-1)
            if t < T - 1:                            # the last one's is in `end`
                dots[:, t] -= (b * yK * v[:, t]).sum(-1)
        else:
            dots[:, t] = (dO[:, t] * (old[t] + b * p * (v[:, t] - kS[t]))).sum(-1) - (dv * v[:, t]).sum(-1)
        Y = a[:, t, :, None, None] * (Y + scale * q[:, t, :, :, None] * dO[:, t, :, None] - k[:, t, :, :, None] * dv[:, :, None])
    # the parts are in `dtype`, their sum in 64 bits, as the kernel's
    return dots.double().flip(1).cumsum(1).flip(1) + total.double()[:, None]


def errors(x, dO, dS_T, dtype, kept):
    want = ref.backward(*(x[n] for n in ("q", "k", "v", "g", "beta", "scale")), dO, x["S0"], dS_T)[0]["dg"]
    return ((sums(x, dO, dS_T, dtype, kept).double() - want).norm(dim=1) / want.norm(dim=1)).amax(0)


@pytest.mark.parametrize("seed", [0, 1])
def test_summands_that_keep_the_decay(seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    B, T, d, dv = 2, 100, 32, 32
    rates = (0.01, 0.3, 3.0, 5.0, 10.0, 20.0)
    H = len(rates)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    x = dict(q=unit(r(B, T, H, d)), k=unit(r(B, T, H, d)), v=r(B, T, H, dv), beta=torch.sigmoid(r(B, T, H)),
             g=-torch.tensor(rates) * (1.0 + 0.1 * r(B, T, H)).clamp(0.5, 1.5), scale=d ** -0.5, S0=r(B, H, d, dv))
    dO, dS_T = r(B, T, H, dv), r(B, H, d, dv)
    assert (errors(x, dO, dS_T, torch.float64, True) < 1e-9).all()          # the same sum
    assert (errors(x, dO, dS_T, torch.float64, False)[:4] < 1e-9).all()
    kept, lost = errors(x, dO, dS_T, torch.float32, True), errors(x, dO, dS_T, torch.float32, False)
    print(kept, lost)
    assert (kept < 4e-6).all()
    assert (lost[:2] < 4e-6).all() and (lost[2:] > 4e-6).all() and lost[5] > 1.0
