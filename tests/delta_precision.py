"""How far results of the gated delta rule may be from 64 bits in norm, each head by its own, and a
CPU model of the kernels' chunk form with matrix operands as sums of N bf16 terms, which shows what
the limits tell apart."""
import torch

from linear_precision import product, terms

# fp32 results, and of bf16 inputs the states, dbeta and dS0.  Three bf16 terms hold an operand's 24
# bits and a product of two such leaves out what is below 2^-24, so that fp32 additions remain: some
# hundred of up to 2^-24 (6e-8) each, at random, 2e-7 to 6e-7 of a head's norm (the system's inverse,
# with entries near 1, does not enlarge them).  One operand held in two terms instead is off by up to
# 2^-17 (7.6e-6), 2e-6 and more of a result's norm.
LIMIT = 1e-6

# A bf16 rounding is off by at most half a step, 2^-9 to 2^-8 of the value, and evenly distributed
# below that: between 1.1e-3 and 2.3e-3 in norm, 1.7e-3 over values of all sizes.  o and dv have
# their own alone (o's operands in two terms leave out 2^-17), dq and dk their own and those of the
# states and their gradients, in two parts of dk.  An output off by 1 % is beyond all of them; so is o
# with its pairs' weights in one term, where queries and keys have most of their length in common: what
# the tokens write nearly cancels then, and o is off by up to 9e-3.
OWN = 2.3e-3
LIMITS = dict(o=OWN, dv=OWN, dq=3.0 ** 0.5 * OWN, dk=3.0 ** 0.5 * OWN)

CHUNK = 64
OPERANDS = ("rows", "state", "inverse", "system", "weights", "written", "update", "back_state", "back_weights",
            "back_inverse", "back_system", "back_update", "qk_states", "qk_written", "qk_pairs")


def limit(name, dtype):
    """dg's is in test_gpu_delta_gates."""
    return LIMITS.get(name, LIMIT) if dtype == torch.bfloat16 else LIMIT


def errors(got, want, heads):
    """The largest error in norm of a head: |got - want| / |want| over all of its elements.  heads:
    the dimension that counts them."""
    got, want = (t.detach().double().cpu().movedim(heads, 0).flatten(1) for t in (got, want))
    return float(((got - want).norm(dim=1) / want.norm(dim=1)).max())


def inputs(B, T, H, Hk, dk, dv, dtype, seed, queries=False):
    """On the CPU: queries and keys of length 1, the keys of a head (and the queries) with most of
    their length in common, so that the inverses (and the pairs' weights) are far from zero; half-lives
    from one token to 350; states that do not hide what the tokens write."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)  # noqa: E731
    common = 2.0 * unit(r(1, 1, Hk, dk))
    x = dict(q=unit(unit(r(B, T, Hk, dk)) + queries * common), k=unit(unit(r(B, T, Hk, dk)) + common), v=r(B, T, H, dv), dO=r(B, T, H, dv))
    x = {n: t.to(dtype) for n, t in x.items()}
    rate = torch.exp2(-9.0 * torch.arange(H) / max(H - 1, 1))
    x.update(g=-rate * r(B, T, H).abs(), beta=torch.sigmoid(r(B, T, H)), scale=dk ** -0.5, S0=0.1 * r(B, H, dk, dv),
             dS_T=0.1 * r(B, H, dk, dv))
    return x


def model(x, **fewer):
    """{o, S_T, dq, dk, dv, dbeta, dS0} of the chunk form before their rounding, every operand in three
    terms but those named.  bf16: o's and dq's and dk's operands as the kernels have them."""
    n = dict.fromkeys(OPERANDS, 3)
    if x["q"].dtype == torch.bfloat16:
        n.update(rows=1, weights=2, written=2, qk_states=1, qk_written=2, qk_pairs=2)
    n.update(fewer)
    H, T, scale = x["v"].shape[2], x["v"].shape[1], x["scale"]
    heads = lambda t: t.float().repeat_interleave(H // t.shape[2], dim=2).transpose(1, 2)  # noqa: E731
    q, k, v, dO = heads(x["q"]), heads(x["k"]), heads(x["v"]), heads(x["dO"])
    g, beta = x["g"].transpose(1, 2), x["beta"].transpose(1, 2)
    T_ = lambda a: [t.transpose(-1, -2) for t in a]  # noqa: E731
    S, Y, kept = x["S0"].clone(), x["dS_T"].clone(), []
    o, dq, dk, dv, dbeta = (torch.empty_like(t) for t in (v, q, k, v, beta))
    for t in range(0, T, CHUNK):
        at = slice(t, t + CHUNK)
        qc, kc, dc = (terms(y[:, :, at], n["rows"]) for y in (q, k, dO))
        b, G = beta[:, :, at, None], g[:, :, at].double().cumsum(-1)
        c = G.shape[-1]
        D = torch.tril(torch.exp((G[..., :, None] - G[..., None, :]).clamp(max=0))).float()
        grow, end = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
        N = torch.tril(product(kc, T_(kc)) * D, -1)
        eye = torch.eye(c).expand_as(N)
        inv = torch.linalg.solve_triangular(eye + N * b.mT, eye, upper=False)
        invt = torch.linalg.solve_triangular(eye + b * N, eye, upper=False).mT
        qk = product(qc, T_(kc)) * D * scale
        R = v[:, :, at] - grow * product(kc, terms(S, n["state"]))
        E = product(terms(inv, n["inverse"]), terms(R, n["system"]))
        o[:, :, at] = scale * grow * product(qc, terms(S, n["state"])) + product(terms(qk * b.mT, n["weights"]), terms(E, n["written"]))
        kept.append((at, qc, kc, dc, b, grow, end, invt, qk.mT, E, torch.exp(G[..., -1]).float()[..., None, None], S, D))
        S = torch.exp(G[..., -1]).float()[..., None, None] * S + product(T_(kc), terms(end * b * E, n["update"]))
    for at, qc, kc, dc, b, grow, end, invt, qkt, E, decay, S0, D in reversed(kept):
        dU = product(terms(qkt, n["back_weights"]), dc) + end * product(kc, terms(Y, n["back_state"]))
        Z = product(terms(invt, n["back_inverse"]), terms(dU, n["back_system"]))
        dv[:, :, at], dbeta[:, :, at] = b * Z, (Z * E).sum(-1)
        u, r = terms(b * E, n["qk_written"]), terms(b * Z, n["qk_written"])
        Sx, Yx = T_(terms(S0, n["qk_states"])), T_(terms(Y, n["qk_states"]))
        W, X = scale * D * product(dc, T_(u)), torch.tril(D * product(r, T_(u)), -1)
        pairs = lambda w: terms(w, n["qk_pairs"])  # noqa: E731
        dq[:, :, at] = scale * grow * product(dc, Sx) + product(pairs(W), kc)
        dk[:, :, at] = (end * product(u, Yx) - grow * product(r, Sx) + product(pairs(W.mT), qc)
                        - product(pairs(X + X.mT), kc))
        Y = (decay * Y + product(T_(qc), terms(scale * grow * sum(reversed(dc)), n["back_update"]))
             - product(T_(kc), terms(grow * b * Z, n["back_update"])))
    back = lambda t: t.transpose(1, 2)  # noqa: E731
    shared = lambda t: back(t).unflatten(2, x["q"].shape[2:3] + (-1,)).sum(3)  # noqa: E731
    return dict(o=back(o), S_T=S, dq=shared(dq), dk=shared(dk), dv=back(dv), dbeta=back(dbeta), dS0=Y)
