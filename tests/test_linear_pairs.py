"""The sums over pairs of tokens (CPU) against the token-by-token definitions."""
import pytest
import torch

import linear_pairs as pairs
import linear_ref as ref


def _close(a, b):
    assert a.shape == b.shape and torch.allclose(a, b, rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("B,T,H,Hk,dk,dv,ragged,state", [
    (1, 1, 1, 1, 3, 2, False, False), (2, 9, 4, 2, 5, 3, True, True), (3, 6, 2, 1, 4, 4, True, False),
    (1, 12, 3, 3, 2, 6, False, True)])
def test_prefill_and_gradients(B, T, H, Hk, dk, dv, ragged, state):
    gen = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k, v, dO = r(B, T, Hk, dk), r(B, T, Hk, dk), r(B, T, H, dv), r(B, T, H, dv)
    g = -torch.rand(H, generator=gen)
    g[0] = float("-inf")
    S0, dS = (r(B, H, dk, dv), r(B, H, dk, dv)) if state else (None, None)
    lens = torch.tensor([T // 2, 0, T + 3][:B], dtype=torch.int32) if ragged else None
    for a, b in zip(pairs.prefill(q, k, v, g, 0.7, S0, lens), ref.prefill(q, k, v, g, 0.7, S0, lens)[:2]):
        _close(a, b)
    got, want = (m.backward(q, k, v, g, 0.7, dO, S0, dS, lens) for m in (pairs, ref))
    for n in want:
        _close(got[n], want[n])


def test_tree():
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    B, T, H, Hk = 3, 9, 4, 2
    q, k, v, S = r(B, T, Hk, 5), r(B, T, Hk, 5), r(B, T, H, 3), r(B, H, 5, 3)
    g = -torch.rand(H, generator=gen)
    parent = torch.tensor([[-1, 0, 0, 1, 2, -1, 5, 3, 6], [-2, 0, -1, 2, 3, 9, 5, -1, 7],
                           [-1, 1, 0, 2, 3, 4, 5, 6, 7]], dtype=torch.int32)
    _close(pairs.tree(q, k, v, g, 0.3, S, parent), ref.tree(q, k, v, g, 0.3, S, parent))
