"""Plain 64-bit forms of the gated delta rule, of its gradients, of the gated norm and of the
norms between blocks, from their definitions (CPU tensors, torch float64), with the magnitudes
that rounding errors are relative to."""
from __future__ import annotations

import torch

from linear_ref import HALF, MIN_G, _share, f64, lengths

#: Tokens over which a state enters an output as a sum over tokens: a chunk of the prefill and of
#: the gradients.
SPAN = 64


def prefill(q, k, v, g, beta, scale, S0=None, lens=None):
    """A dict: o (zeros past the lengths), S_T; o_mag, what products in fewer bits are relative
    to: |S| at a span's start and |k_j| |beta_j e_j| behind it, times |q|; o_sum and S_sum, what
    one fp32 rounding of a state's column reaches (keys of length 1 and beta in [0, 2] do not
    let it grow); and for the gradients, per sequence and token, the state before it, its
    magnitude after it, and e."""
    B, T, H, dv = v.shape
    q, k, v, beta = _share(q, H), _share(k, H), f64(v), f64(beta)
    a = torch.exp(torch.clamp(f64(g), min=MIN_G))
    z = dict(dtype=torch.float64)
    out = dict(o=torch.zeros(B, T, H, dv, **z), o_mag=torch.zeros(B, T, H, dv, **z), o_sum=torch.zeros(B, T, H, dv, **z),
               S_T=torch.zeros(B, H, q.shape[-1], dv, **z), S_sum=torch.zeros(B, H, q.shape[-1], dv, **z),
               before=[], mag=[], e=[], col=[])
    for b, n in enumerate(lengths(lens, B, T)):
        S = torch.zeros_like(out["S_T"][b]) if S0 is None else f64(S0[b])
        M, col = S.abs(), S.norm(dim=1)
        before, mags, es = [], [], []
        for t in range(n):
            if t % SPAN == 0:
                M = S.abs()
            before.append(S)
            at, kt, bt = a[b, t][:, None, None], k[b, t][:, :, None], beta[b, t][:, None]
            e = v[b, t] - (kt * (at * S)).sum(1)
            S = at * S + kt * (bt * e)[:, None]
            M = at * M + kt.abs() * (bt * e).abs()[:, None]
            # the most that a column has held so far, decayed as its errors are
            col = torch.maximum(at[..., 0] * col, S.norm(dim=1) + v[b, t].abs() + e.abs())
            out["o"][b, t] = scale * (q[b, t][:, :, None] * S).sum(1)
            out["o_mag"][b, t] = abs(scale) * (q[b, t].abs()[:, :, None] * M).sum(1)
            out["o_sum"][b, t] = abs(scale) * q[b, t].norm(dim=1)[:, None] * col
            mags.append(M)
            es.append(e)
        out["S_T"][b], out["S_sum"][b] = S, col[:, None].expand_as(S)
        for name, x in (("before", before), ("mag", mags), ("e", es), ("col", col)):
            out[name].append(x)
    return out


def backward(q, k, v, g, beta, scale, dO, S0=None, dS_T=None, lens=None):
    """(gradients, magnitudes for operands in fewer bits, magnitudes for fp32 sums): dicts; zeros
    past the lengths."""
    B, T, H, dvn = v.shape
    Hk, dkn = q.shape[-2:]
    fwd = prefill(q, k, v, g, beta, scale, S0, lens)
    qs, ks, v, beta, dO = _share(q, H), _share(k, H), f64(v), f64(beta), scale * f64(dO)
    a = torch.exp(torch.clamp(f64(g), min=MIN_G))
    z = dict(dtype=torch.float64)

    def new():
        return dict(dq=torch.zeros(B, T, H, dkn, **z), dk=torch.zeros(B, T, H, dkn, **z), dv=torch.zeros(B, T, H, dvn, **z),
                    dg=torch.zeros(B, T, H, **z), dbeta=torch.zeros(B, T, H, **z), dS0=torch.zeros(B, H, dkn, dvn, **z))

    out, mag, sums = new(), new(), new()
    for b, n in enumerate(lengths(lens, B, T)):
        Y = torch.zeros(H, dkn, dvn, **z) if dS_T is None else f64(dS_T[b])
        N, col, scol = Y.abs(), Y.norm(dim=1), fwd["col"][b]
        token = torch.zeros(H, **z)
        for t in reversed(range(n)):
            if t % SPAN == SPAN - 1:
                N = Y.abs()
            S, at, kt, bt, e = fwd["before"][b][t], a[b, t][:, None, None], ks[b, t], beta[b, t][:, None], fwd["e"][b][t]
            after = at * S + kt[:, :, None] * (bt * e)[:, None]
            R = Y + qs[b, t][:, :, None] * dO[b, t][:, None]
            M = N + qs[b, t].abs()[:, :, None] * dO[b, t].abs()[:, None]
            zt = (kt[:, :, None] * R).sum(1)
            dv = bt * zt
            col = torch.maximum(col, R.norm(dim=1) + dO[b, t].abs() + dv.abs())
            out["dq"][b, t] = (after * dO[b, t][:, None]).sum(2)
            out["dv"][b, t], out["dbeta"][b, t] = dv, (zt * e).sum(1)
            out["dk"][b, t] = (R * (bt * e)[:, None]).sum(2) - (at * S * dv[:, None]).sum(2)
            Y = at * (R - kt[:, :, None] * dv[:, None])
            N = at * (M + kt.abs()[:, :, None] * dv.abs()[:, None])
            out["dg"][b, t] = (Y * S).sum((1, 2))
            before = fwd["mag"][b][t]                       # holds a |S| too
            mag["dq"][b, t] = (before * dO[b, t].abs()[:, None]).sum(2)
            mag["dk"][b, t] = (M * (bt * e).abs()[:, None]).sum(2) + (before * dv.abs()[:, None]).sum(2)
            sums["dq"][b, t] = (scol * dO[b, t].abs()).sum(1)[:, None]
            sums["dk"][b, t] = (col * (bt * e).abs() + scol * (dv.abs() + bt.abs() * col)).sum(1)[:, None]
            sums["dv"][b, t] = bt.abs() * col
            sums["dbeta"][b, t] = (col * e.abs() + zt.abs() * scol).sum(1)
            token = token + (dO[b, t] * (qs[b, t][:, :, None] * after).sum(1)).abs().sum(1) + (dv * v[b, t]).abs().sum(1)
            sums["dg"][b, t] = token + (col * scol).sum(1)
        out["dS0"][b], sums["dS0"][b] = Y, col[:, None].expand_as(Y)
    for d in (out, mag, sums):
        for x in ("dq", "dk"):
            d[x] = d[x].reshape(B, T, Hk, H // Hk, dkn).sum(3)
    return out, mag, sums


def decode(q, k, v, g, beta, scale, S):
    x = prefill(q[:, None], k[:, None], v[:, None], g[:, None], beta[:, None], scale, S)
    return {n: t[:, 0] if n.startswith("o") else t for n, t in x.items()}


def check(name, got, ref, mag, sums, roundings, terms):
    """|got - ref| <= half a step of the result, half a bf16 step of each of `roundings` operands
    on the sum of magnitudes `mag`, and 2^-24 for each of `terms` fp32 roundings on `sums`."""
    half = HALF[got.dtype]
    got, ref = f64(got), f64(ref)
    tol = half * ref.abs() + 1e-37
    if roundings:
        tol = tol + roundings * HALF[torch.bfloat16] * 1.02 * mag
    tol = tol + terms * 2.0 ** -24 * sums
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = int(torch.argmax(torch.where(bad, ((got - ref).abs() / tol).nan_to_num(1e30), torch.zeros(()).double())))
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: got "
                             f"{got.flatten()[i]:.9g}, expected {ref.flatten()[i]:.9g}, tolerance {tol.flatten()[i]:.3g}")


# ----------------------------------------------------------------- norms

def sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def gate(z, act):
    """(the gate, its derivative)"""
    s, rest = sigmoid(z), sigmoid(-z)
    return (s, s * rest) if act == "sigmoid" else (z * s, s * (1.0 + z * rest))


def length(x, eps):
    return torch.sqrt(x.square().mean(-1, keepdim=True) + eps)


def norm_grad(x, dn, eps):
    """(the gradient of x in x / length(x), its magnitude)"""
    r = 1.0 / length(x, eps)
    n = x * r
    return (r * (dn - n * (n * dn).mean(-1, keepdim=True)),
            r * (dn.abs() + n.abs() * (n * dn).abs().mean(-1, keepdim=True)))


def gated_norm(x, z, w, act, eps):
    x, z = f64(x), f64(z)
    y = x / length(x, eps) * gate(z, act)[0]
    return y if w is None else y * f64(w)


def gated_norm_backward(x, z, w, dy, act, eps):
    """({dx, dz, dw}, their magnitudes)"""
    x, z, dy = f64(x), f64(z), f64(dy)
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else f64(w)
    n, (a, da) = x / length(x, eps), gate(z, act)
    dx, mx = norm_grad(x, dy * a * w, eps)
    lead = tuple(range(x.dim() - 1))
    s, rest = sigmoid(z), sigmoid(-z)
    mz = da.abs() if act == "sigmoid" else s * (1.0 + (z * rest).abs())
    return (dict(dx=dx, dz=dy * n * w * da, dw=(dy * a * n).sum(lead)),
            dict(dx=mx, dz=(dy * n * w).abs() * mz, dw=(dy * a * n).abs().sum(lead)))


def block_norm(y, r, z, w_y, w_n, norm_y, scale, eps):
    """({h, n}, their magnitudes)"""
    r = f64(r)
    u = torch.zeros_like(r)
    if y is not None:
        u = f64(y) / length(f64(y), eps) if norm_y else f64(y)
        u = scale * u * (1.0 if w_y is None else f64(w_y)) * (1.0 if z is None else sigmoid(f64(z)))
    h, w = r + u, 1.0 if w_n is None else f64(w_n)
    m = r.abs() + u.abs()
    n = h / length(h, eps) * w
    # an error of h by m's share reaches n itself and through the row's length
    reach = (m + h.abs() / length(h, eps) * length(m, eps)) / length(h, eps) * abs(w)
    return dict(h=h, n=n), dict(h=m, n=reach)


def block_norm_backward(y, h, dn, dh, z, w_y, w_n, norm_y, scale, eps):
    """({dr, dy, dz, dw_y, dw_n}, their magnitudes; None where there is no input)"""
    h, dn = f64(h), f64(dn)
    w_n1 = 1.0 if w_n is None else f64(w_n)
    dr, mr = norm_grad(h, dn * w_n1, eps)
    if dh is not None:
        dr, mr = dr + f64(dh), mr + f64(dh).abs()
    lead = tuple(range(h.dim() - 1))
    k = dn * h / length(h, eps)
    out = dict(dr=dr, dy=None, dz=None, dw_y=None, dw_n=None if w_n is None else k.sum(lead))
    mag = dict(dr=mr, dy=None, dz=None, dw_y=None, dw_n=k.abs().sum(lead))
    if y is None:
        return out, mag
    y = f64(y)
    m = y / length(y, eps) if norm_y else y
    w = 1.0 if w_y is None else f64(w_y)
    a, rest = (1.0, 0.0) if z is None else (sigmoid(f64(z)), sigmoid(-f64(z)))
    du, mu = scale * dr, abs(scale) * mr
    dm, mm = du * a * w, mu * a * abs(w)
    if norm_y:
        out["dy"], mag["dy"] = norm_grad(y, dm, eps)[0], norm_grad(y, mm, eps)[1]
    else:
        out["dy"], mag["dy"] = dm, mm
    if z is not None:
        out["dz"], mag["dz"] = dm * m * rest, mm * m.abs() * rest
    if w_y is not None:
        out["dw_y"], mag["dw_y"] = (du * a * m).sum(lead), (mu * a * m.abs()).sum(lead)
    return out, mag


def check_sums(name, got, ref, mag, terms):
    """|got - ref| <= half a step of the result + 2^-24 for each of `terms` fp32 roundings on mag."""
    h = HALF[got.dtype]
    got, ref = f64(got), f64(ref)
    tol = h * ref.abs() + terms * 2.0 ** -24 * f64(mag) + 1e-37
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = int(torch.argmax(torch.where(bad, ((got - ref).abs() / tol).nan_to_num(1e30), torch.zeros(()).double())))
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: got "
                             f"{got.flatten()[i]:.9g}, expected {ref.flatten()[i]:.9g}, tolerance {tol.flatten()[i]:.3g}")
