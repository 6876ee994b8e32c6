"""How far fp32 results of linear attention, and states of either type, may be from 64 bits in
norm, and a CPU model of the kernel's chunk form with matrix operands as sums of N bf16 terms,
which shows what the limit tells apart."""
import torch

# Three bf16 terms hold an operand's 24 bits; of a product of two such the terms below 2^-24 are
# left out.  What remains is fp32 addition: a result has some hundred roundings of at most 2^-24
# (6e-8) of a partial sum each, at random, which add up to a few of them in norm (1e-7 to
# 4e-7).  With two terms an operand is off by up to 2^-17 (7.6e-6), which is 2e-6 to 4e-6 of a
# result's norm.  The limit lies between, a factor of two from either.
LIMIT = 1e-6

CHUNK = 32


def error(got, want):
    got, want = got.detach().double().cpu(), want.double().cpu()
    return float(torch.linalg.vector_norm(got - want) / torch.linalg.vector_norm(want))


def inputs(B, T, H, Hk, dk, dv, dtype, seed):
    """On the CPU: rows of queries and keys of length 1, half-lives from one token to 350."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)  # noqa: E731
    x = dict(q=unit(r(B, T, Hk, dk)), k=unit(r(B, T, Hk, dk)), v=r(B, T, H, dv), dO=r(B, T, H, dv))
    x = {n: t.to(dtype) for n, t in x.items()}
    x.update(g=-torch.exp2(-9.0 * torch.rand(H, generator=gen)), scale=dk ** -0.5, S0=r(B, H, dk, dv),
             dS_T=r(B, H, dk, dv))
    return x


def terms(x, n):
    """fp32 values as n bf16 ones (each what the ones before leave, rounded) in fp32"""
    out = []
    for _ in range(n):
        out.append(x.bfloat16().float())
        x = x - out[-1]
    return out


def product(a, b):
    """Of operands as terms: the products down to 2^-24 of the largest, small ones first"""
    c = None
    for s in reversed(range(min(len(a) + len(b) - 2, 2) + 1)):
        for i in range(len(a)):
            if 0 <= s - i < len(b):
                p = a[i] @ b[s - i]
                c = p if c is None else c + p
    return c


def model(x, rows, weights, update):
    """(o, S_T) of the chunk form: q, k and v as `rows` terms, the state and the pair weights as
    `weights`, v times its decays in the state's update as `update`."""
    H, T = x["v"].shape[2], x["v"].shape[1]
    heads = lambda t: t.float().repeat_interleave(H // t.shape[2], dim=2).transpose(1, 2)  # noqa: E731
    q, k, v = heads(x["q"]), heads(x["k"]), heads(x["v"])
    g, scale, S = x["g"][:, None], x["scale"], x["S0"].clone()
    o = torch.empty_like(v)
    for t in range(0, T, CHUNK):
        qc, kc, vc = (terms(y[:, :, t:t + CHUNK], rows) for y in (q, k, v))
        c = qc[0].shape[2]
        i = torch.arange(c)
        gap = i[:, None] - i
        W = torch.where(gap >= 0, scale * torch.exp(g[..., None] * gap.clamp(min=0)), 0.0)
        P = product(qc, [y.transpose(-1, -2) for y in kc]) * W
        o[:, :, t:t + c] = (scale * torch.exp(g * (i + 1)))[..., None] * product(qc, terms(S, weights)) + product(
            terms(P, weights), vc)
        u = terms(sum(reversed(vc)) * torch.exp(g * (c - 1 - i))[..., None], update)
        S = torch.exp(g * c)[..., None] * S + product([y.transpose(-1, -2) for y in kc], u)
    return o.transpose(1, 2), S
