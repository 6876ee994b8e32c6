"""Linear attention with a decay for each head, its gradients and draft trees in 64 bits as sums
over pairs of tokens, for sizes where the token-by-token forms of ``linear_ref`` take too long.
Runs on the tensors' device (which must compute in float64); the same sums of products, so on absolute values each gives
the magnitude that rounding errors are relative to."""
import torch

from linear_ref import MIN_G


def _f64(x):
    return None if x is None else x.detach().double()


def _heads(x, H):
    """[B, T, h, d] -> [B, H, T, d] in 64 bits, a shared head repeated"""
    return _f64(x).repeat_interleave(H // x.shape[2], dim=2).transpose(1, 2).contiguous()


def _t(x):
    return x.transpose(-1, -2).contiguous()


def _setup(q, k, v, g, lens):
    B, T, H, _ = v.shape
    n = torch.full((B,), T, device=v.device) if lens is None else lens.long().clamp(0, T)
    t = torch.arange(T, device=v.device)
    live = t < n[:, None]
    lg = torch.clamp(_f64(g), min=MIN_G)[:, None]
    gap = t[:, None] - t
    W = torch.where(gap >= 0, torch.exp(lg[..., None] * gap.clamp(min=0)), 0.0)                    # [H, T, T]
    first = torch.exp(lg * (t + 1))[None, ..., None]                                               # [1, H, T, 1]
    behind = torch.where(live[:, None], torch.exp(lg * (n[:, None, None] - 1 - t).clamp(min=0)), 0.0)[..., None]
    whole = torch.exp(lg * n[:, None, None])[..., None]                                            # [B, H, 1, 1]
    m = live[:, None, :, None]
    take = lambda x: torch.where(m, _heads(x, H), 0.0)  # noqa: E731
    return take, W, first, behind, whole, m


def prefill(q, k, v, g, scale, S0=None, lens=None):
    """(o with zeros past the lengths, S_T)"""
    take, W, first, behind, whole, m = _setup(q, k, v, g, lens)
    q, k, v = take(q), take(k), take(v)
    o = ((q @ _t(k)) * W) @ v
    S_T = _t(behind * k) @ v
    if S0 is not None:
        o = o + first * (q @ _f64(S0))
        S_T = S_T + whole * _f64(S0)
    return (scale * o).transpose(1, 2), S_T


def backward(q, k, v, g, scale, dO, S0=None, dS_T=None, lens=None):
    """Gradients of sum(dO o) + sum(dS_T S_T) (zeros past the lengths)"""
    B, T, Hk, d = q.shape
    H = v.shape[2]
    take, W, first, behind, whole, m = _setup(q, k, v, g, lens)
    q, k, v, dO = take(q), take(k), take(v), take(dO)
    X, P = scale * (dO @ _t(v)) * W, scale * (q @ _t(k)) * W
    dq, dk, dv = X @ k, _t(X) @ q, _t(P) @ dO
    dS0 = scale * (_t(first * q) @ dO)
    if S0 is not None:
        dq = dq + scale * torch.where(m, first, 0.0) * (dO @ _t(_f64(S0)))
    if dS_T is not None:
        end = _f64(dS_T)
        dk, dv, dS0 = dk + behind * (v @ _t(end)), dv + behind * (k @ end), dS0 + whole * end
    fold = lambda x: x.transpose(1, 2).reshape(B, T, Hk, H // Hk, d).sum(3)  # noqa: E731
    return dict(dq=fold(dq), dk=fold(dk), dv=dv.transpose(1, 2), dS0=dS0)


def tree(q, k, v, g, scale, S, parent):
    """Outputs of the tree's nodes (zeros for absent ones)"""
    B, T, H, _ = v.shape
    on = torch.zeros(B, T, T + 1, dtype=torch.float64)              # [b, i, j]: j is i or above it (T: S)
    for b, row in enumerate(parent.tolist()):
        for i, p in enumerate(row):
            if p == -1:
                on[b, i, T] = 1
            elif 0 <= p < i:
                on[b, i] = on[b, p]
            on[b, i, i] = 1
    on = on.to(v.device)
    top, on = on[..., T], on[..., :T]
    depth = on.sum(2)
    lg = torch.clamp(_f64(g), min=MIN_G)[:, None]
    gap = (depth[:, :, None] - depth[:, None]).clamp(min=0)[:, None]
    W = on[:, None] * torch.exp(lg[..., None] * gap)
    q, k, v = _heads(q, H), _heads(k, H), _heads(v, H)
    o = ((q @ _t(k)) * W) @ v + torch.exp(lg * depth[:, None])[..., None] * (q @ _f64(S))
    return (scale * top[:, None, :, None] * o).transpose(1, 2)
