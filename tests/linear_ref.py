"""Plain 64-bit forms of linear attention with a decay for each head, of its
gradients, of draft trees over its states and of the norm with the position
rotation, token by token from their definitions (CPU tensors, torch float64).

Every form is a sum of products, so called on absolute values it gives the
magnitude that rounding errors are relative to."""
from __future__ import annotations

import torch

MIN_G = -1e4     # log-decays below this are taken as this


def f64(x):
    return None if x is None else x.detach().double().cpu()


def _decay(g):
    return torch.exp(torch.clamp(f64(g), min=MIN_G))


def _share(x, H):
    """[..., Hk, d] -> [..., H, d]"""
    return f64(x).repeat_interleave(H // x.shape[-2], dim=-2)


def lengths(lens, B, T):
    return [T] * B if lens is None else [min(max(int(n), 0), T) for n in lens]


def prefill(q, k, v, g, scale, S0=None, lens=None):
    """(o with zeros past the lengths, S_T, states before each token)"""
    B, T, H, dv = v.shape
    q, k, v, a = _share(q, H), _share(k, H), f64(v), _decay(g)[:, None, None]
    o = torch.zeros(B, T, H, dv, dtype=torch.float64)
    S_T = torch.zeros(B, H, q.shape[-1], dv, dtype=torch.float64)
    before = []
    for b, n in enumerate(lengths(lens, B, T)):
        S = torch.zeros_like(S_T[b]) if S0 is None else f64(S0[b])
        before.append([])
        for t in range(n):
            before[b].append(S)
            S = a * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            o[b, t] = scale * (q[b, t][:, None, :] @ S)[:, 0]
        S_T[b] = S
    return o, S_T, before


def backward(q, k, v, g, scale, dO, S0=None, dS_T=None, lens=None):
    """Gradients by the reverse recurrence (dict; zeros past the lengths)."""
    B, T, H, dv_ = v.shape
    Hk, dk_ = q.shape[-2:]
    _, _, before = prefill(q, k, v, g, scale, S0, lens)
    qs, ks, v, dO, a = _share(q, H), _share(k, H), f64(v), f64(dO), _decay(g)[:, None, None]
    z = dict(dtype=torch.float64)
    dq, dk, dv = torch.zeros(B, T, H, dk_, **z), torch.zeros(B, T, H, dk_, **z), torch.zeros(B, T, H, dv_, **z)
    dS0 = torch.zeros(B, H, dk_, dv_, **z)
    for b, n in enumerate(lengths(lens, B, T)):
        Y = torch.zeros(H, dk_, dv_, **z) if dS_T is None else f64(dS_T[b])
        for t in reversed(range(n)):
            S = a * before[b][t] + ks[b, t][:, :, None] * v[b, t][:, None, :]
            R = scale * qs[b, t][:, :, None] * dO[b, t][:, None, :] + Y
            dq[b, t] = scale * (S @ dO[b, t][:, :, None])[:, :, 0]
            dk[b, t] = (R @ v[b, t][:, :, None])[:, :, 0]
            dv[b, t] = (ks[b, t][:, None, :] @ R)[:, 0]
            Y = a * R
        dS0[b] = Y
    fold = lambda x: x.reshape(B, T, Hk, H // Hk, dk_).sum(3)  # noqa: E731
    return dict(dq=fold(dq), dk=fold(dk), dv=dv, dS0=dS0)


def decode(q, k, v, g, scale, S):
    o, S_T, _ = prefill(q[:, None], k[:, None], v[:, None], g, scale, S)
    return o[:, 0], S_T


def tree_states(k, v, g, S, parent):
    """For each sequence a dict node -> state after it (-1: S); absent nodes have none."""
    B, T, H, _ = v.shape
    k, v, a = _share(k, H), f64(v), _decay(g)[:, None, None]
    out = []
    for b in range(B):
        st = {-1: f64(S[b])}
        for t in range(T):
            p = int(parent[b, t])
            if -1 <= p < t and p in st:
                st[t] = a * st[p] + k[b, t][:, :, None] * v[b, t][:, None, :]
        out.append(st)
    return out


def tree(q, k, v, g, scale, S, parent):
    st = tree_states(k, v, g, S, parent)
    qs = _share(q, v.shape[2])
    o = torch.zeros(v.shape, dtype=torch.float64)
    for b, nodes in enumerate(st):
        for t, M in nodes.items():
            if t >= 0:
                o[b, t] = scale * (qs[b, t][:, None, :] @ M)[:, 0]
    return o


def commit(k, v, g, S, parent, accepted, S_out):
    """S_out with the committed states in it (skipped sequences keep theirs)."""
    out = f64(S_out).clone()
    for b, nodes in enumerate(tree_states(k, v, g, S, parent)):
        if int(accepted[b]) in nodes:
            out[b] = nodes[int(accepted[b])]
    return out


def _c(norm, d):
    return 1.0 if norm == "l2" else 1.0 / d


def _turn(x, positions, inv_freq, interleaved, sign, mag=False):
    """Pairs turned by sign * angle; with mag: the sum of the two terms' magnitudes."""
    if inv_freq is None:
        return x.clone()
    rot = 2 * inv_freq.numel()
    ang = positions.double().cpu()[:, :, None, None] * inv_freq.double().cpu()
    cos, sin = torch.cos(ang), sign * torch.sin(ang)
    y = x.clone()
    i = torch.arange(rot // 2)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[..., first], x[..., second]
    if mag:
        y[..., first] = y[..., second] = a.abs() + b.abs()
    else:
        y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    return y


def norm_rope(x, w, positions, inv_freq, norm, eps, interleaved):
    """(y, the magnitude its rounding is relative to)"""
    x = f64(x)
    u = x / torch.sqrt(_c(norm, x.shape[-1]) * (x * x).sum(-1, keepdim=True) + eps)
    u = u if w is None else u * f64(w)
    return (_turn(u, positions, inv_freq, interleaved, 1.0),
            _turn(u.abs(), positions, inv_freq, interleaved, 1.0, mag=True))


def norm_rope_backward(x, w, positions, inv_freq, dy, norm, eps, interleaved):
    """(dx, its magnitude, dw, its magnitude)"""
    x, dy = f64(x), f64(dy)
    c = _c(norm, x.shape[-1])
    r = 1.0 / torch.sqrt(c * (x * x).sum(-1, keepdim=True) + eps)
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else f64(w)

    du = _turn(dy, positions, inv_freq, interleaved, -1.0)
    m = _turn(dy.abs(), positions, inv_freq, interleaved, -1.0, mag=True)
    dn, mdn = w * du, w.abs() * m
    dot, mdot = (x * dn).sum(-1, keepdim=True), (x.abs() * mdn).sum(-1, keepdim=True)
    dx = r * dn - c * r**3 * x * dot
    return (dx, r * mdn + c * r**3 * x.abs() * mdot, (du * x * r).sum((0, 1, 2)),
            (m * x.abs() * r).sum((0, 1, 2)))


# ----------------------------------------------------------------- tolerances

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def check(name, got, ref, mag, dtype, roundings, terms):
    """|got - ref| <= half a step of the result
                     + half a step of `dtype` on each of `roundings` operands
                       that are rounded to it inside (relative to the sum of
                       magnitudes `mag`)
                     + 2^-24 `terms` mag for fp32 sums of that many terms."""
    h = HALF[got.dtype]
    got, ref, mag = f64(got), f64(ref), f64(mag)
    tol = h * ref.abs() + (roundings * HALF[dtype] * 1.02 + terms * 2.0 ** -24) * mag + 1e-37
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = int(torch.argmax(torch.where(bad, ((got - ref).abs() / tol).nan_to_num(1e30), torch.zeros(()).double())))
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: got "
                             f"{got.flatten()[i]:.9g}, expected {ref.flatten()[i]:.9g}, "
                             f"tolerance {tol.flatten()[i]:.3g}")
