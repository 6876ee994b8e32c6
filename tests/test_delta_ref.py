"""The plain 64-bit forms of the delta rule and the norms against derivatives by autograd and
against closed forms (CPU)."""
import pytest
import torch

import delta_ref as ref

F64 = torch.float64


def _rand(gen, *s):
    return torch.randn(*s, generator=gen, dtype=F64)


def _inputs(seed, B=2, T=7, H=4, Hk=2, dk=5, dv=3):
    gen = torch.Generator().manual_seed(seed)
    return dict(q=_rand(gen, B, T, Hk, dk), k=0.5 * _rand(gen, B, T, Hk, dk), v=_rand(gen, B, T, H, dv),
                g=-_rand(gen, B, T, H).abs(), beta=torch.sigmoid(_rand(gen, B, T, H)), S0=_rand(gen, B, H, dk, dv)), gen


def _loss(x, dO, dS, lens, scale=0.7):
    """The recurrence in torch operations, for autograd."""
    B, T, H, dv = x["v"].shape
    G = H // x["q"].shape[2]
    q, k = (x[n].repeat_interleave(G, dim=2) for n in ("q", "k"))
    total = 0.0
    for b in range(B):
        S = x["S0"][b]
        for t in range(T if lens is None else lens[b]):
            S = torch.exp(x["g"][b, t])[:, None, None] * S
            e = x["v"][b, t] - (k[b, t][:, :, None] * S).sum(1)
            S = S + x["beta"][b, t][:, None, None] * k[b, t][:, :, None] * e[:, None]
            total = total + scale * ((q[b, t][:, :, None] * S).sum(1) * dO[b, t]).sum()
        total = total + (S * dS[b]).sum()
    return total


@pytest.mark.parametrize("lens", [None, [7, 3], [0, 1]])
def test_delta_gradients_are_autograds(lens):
    x, gen = _inputs(1)
    dO, dS = _rand(gen, *x["v"].shape), _rand(gen, *x["S0"].shape)
    leaves = {n: t.clone().requires_grad_() for n, t in x.items()}
    _loss(leaves, dO, dS, lens).backward()
    got, mag, sums = ref.backward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.7, dO, x["S0"], dS, lens)
    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("S0", "dS0")):
        want = leaves[n].grad
        assert torch.allclose(got[d], torch.zeros_like(x[n]) if want is None else want, rtol=1e-11, atol=1e-12), n
        assert (sums[d] >= 0).all() and (mag[d] >= 0).all()


def test_delta_rule_closed_forms():
    """beta = 1 and a key of length 1: the state then answers that key with that value; beta = 0
    decays only; g = -infinity starts anew."""
    x, _ = _inputs(2, T=3)
    x["k"] = x["k"] / x["k"].norm(dim=-1, keepdim=True)
    one = {**x, "beta": torch.ones_like(x["beta"]), "q": x["k"]}
    out = ref.prefill(one["q"], one["k"], one["v"], one["g"], one["beta"], 1.0, one["S0"])
    assert torch.allclose(out["o"], one["v"], atol=1e-12)
    none = ref.prefill(x["q"], x["k"], x["v"], x["g"], torch.zeros_like(x["beta"]), 1.0, x["S0"])
    assert torch.allclose(none["S_T"], torch.exp(x["g"].sum(1))[..., None, None] * x["S0"], atol=1e-12)
    g = x["g"].clone()
    g[:, 1] = float("-inf")
    cut = ref.prefill(x["q"], x["k"], x["v"], g, x["beta"], 1.0, x["S0"])
    new = ref.prefill(*(x[n][:, 1:] for n in ("q", "k", "v")), g[:, 1:], x["beta"][:, 1:], 1.0)
    assert torch.equal(cut["S_T"], new["S_T"])


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("weighted", [True, False])
def test_gated_norm_gradients_are_autograds(act, weighted):
    gen = torch.Generator().manual_seed(3)
    x, z, dy = (_rand(gen, 4, 6, 8) for _ in range(3))
    w = _rand(gen, 8) if weighted else None
    leaves = [None if t is None else t.clone().requires_grad_() for t in (x, z, w)]
    a = torch.sigmoid(leaves[1]) * (leaves[1] if act == "silu" else 1.0)
    n = leaves[0] * torch.rsqrt(leaves[0].square().mean(-1, keepdim=True) + 1e-3)
    y = n * a if w is None else n * a * leaves[2]
    assert torch.allclose(ref.gated_norm(x, z, w, act, 1e-3), y, atol=1e-13)
    y.backward(dy)
    got, mag = ref.gated_norm_backward(x, z, w, dy, act, 1e-3)
    for d, t in zip(("dx", "dz", "dw"), leaves):
        if t is not None:
            assert torch.allclose(got[d], t.grad, atol=1e-12) and (mag[d] >= got[d].abs() - 1e-12).all(), d


@pytest.mark.parametrize("norm_y", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("weighted", [True, False])
def test_block_norm_gradients_are_autograds(norm_y, gate, weighted):
    gen = torch.Generator().manual_seed(4)
    y, r, dn, dh = (_rand(gen, 5, 8) for _ in range(4))
    z = _rand(gen, 5, 8) if gate else None
    w_y, w_n = (_rand(gen, 8) if weighted else None for _ in range(2))
    leaves = [None if t is None else t.clone().requires_grad_() for t in (y, r, z, w_y, w_n)]
    ly, lr, lz, lw, ln = leaves
    norm = lambda t: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-3)  # noqa: E731
    u = norm(ly) if norm_y else ly
    u = u if lw is None else u * lw
    u = u if lz is None else u * torch.sigmoid(lz)
    h = lr + 0.3 * u
    n = norm(h) if ln is None else norm(h) * ln
    out, mag = ref.block_norm(y, r, z, w_y, w_n, norm_y, 0.3, 1e-3)
    assert torch.allclose(out["h"], h, atol=1e-13) and torch.allclose(out["n"], n, atol=1e-13)
    torch.autograd.backward([h, n], [dh, dn])
    got, mag = ref.block_norm_backward(y, h.detach(), dn, dh, z, w_y, w_n, norm_y, 0.3, 1e-3)
    for d, t in zip(("dy", "dr", "dz", "dw_y", "dw_n"), leaves):
        if t is None:
            assert got[d] is None
        else:
            assert torch.allclose(got[d], t.grad, atol=1e-12) and (mag[d] >= got[d].abs() - 1e-12).all(), d
    first, _ = ref.block_norm(None, r, None, None, w_n, False, 1.0, 1e-3)
    assert torch.equal(first["h"], r)
