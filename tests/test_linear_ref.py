"""The 64-bit forms that the GPU tests compare with, checked on the CPU: the
gradients against differences of the forward form, the tree against the plain
recurrence along each of its paths, the norm's gradients against differences."""
import torch

import linear_ref as ref


def _inputs(B=2, T=5, H=4, Hk=2, dk=3, dv=2, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    return dict(q=r(B, T, Hk, dk), k=r(B, T, Hk, dk), v=r(B, T, H, dv), g=-r(H).abs(),
                S0=r(B, H, dk, dv)), r(B, T, H, dv), r(B, H, dk, dv)


def test_gradients_against_differences():
    x, dO, dS = _inputs()
    lens = [5, 3]

    def loss(x):
        o, S, _ = ref.prefill(x["q"], x["k"], x["v"], x["g"], 0.7, x["S0"], lens)
        return float((o * dO).sum() + (S * dS).sum())

    got = ref.backward(x["q"], x["k"], x["v"], x["g"], 0.7, dO, x["S0"], dS, lens)
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("S0", "dS0")):
        grad = got[key].flatten()
        for i in range(0, x[name].numel(), 3):
            # the loss is linear in each single entry: the difference is exact
            up, down = (dict(x, **{name: x[name].clone()}) for _ in range(2))
            up[name].view(-1)[i] += 1.0
            down[name].view(-1)[i] -= 1.0
            assert abs((loss(up) - loss(down)) / 2 - float(grad[i])) < 1e-9, (name, i)


def test_tree_is_the_recurrence_along_each_path():
    x, _, _ = _inputs(T=7)
    parent = torch.tensor([[-1, 0, 0, 1, -1, 4, 9], [-1, -1, 1, -2, 3, 2, 0]])
    o = ref.tree(x["q"], x["k"], x["v"], x["g"], 0.7, x["S0"], parent)
    paths = {0: {0: [0], 1: [0, 1], 2: [0, 2], 3: [0, 1, 3], 4: [4], 5: [4, 5]},
             1: {0: [0], 1: [1], 2: [1, 2], 5: [1, 2, 5], 6: [0, 6]}}
    for b in (0, 1):
        for t in range(7):
            if t not in paths[b]:
                assert (o[b, t] == 0).all()          # absent, or below an absent node
                continue
            p = paths[b][t]
            y, S, _ = ref.prefill(*(x[n][b:b + 1, p] for n in "qkv"), x["g"], 0.7, x["S0"][b:b + 1])
            assert torch.allclose(o[b, t], y[0, -1], atol=1e-12)
            got = ref.commit(x["k"], x["v"], x["g"], x["S0"], parent, [t, t], x["S0"])
            assert torch.allclose(got[b], S[0], atol=1e-12)


def test_norm_gradients_against_differences():
    gen = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(1, 2, 3, 8, generator=gen, dtype=torch.float64) for _ in range(2))
    w = torch.randn(8, generator=gen, dtype=torch.float64)
    pos, freq = torch.tensor([[5, 70000]]), torch.tensor([1.0, 0.25, 0.001])
    for norm in ("l2", "rms"):
        for il in (False, True):
            f = lambda x, w: float((ref.norm_rope(x, w, pos, freq, norm, 1e-3, il)[0] * dy).sum())  # noqa: E731
            dx, _, dw, _ = ref.norm_rope_backward(x, w, pos, freq, dy, norm, 1e-3, il)
            h = 1e-5
            for i in range(x.numel()):
                up, down = x.clone(), x.clone()
                up.view(-1)[i] += h
                down.view(-1)[i] -= h
                assert abs((f(up, w) - f(down, w)) / (2 * h) - float(dx.flatten()[i])) < 1e-7
            for i in range(8):
                up, down = w.clone(), w.clone()
                up[i] += 1.0
                down[i] -= 1.0
                assert abs((f(x, up) - f(x, down)) / 2 - float(dw[i])) < 1e-9
