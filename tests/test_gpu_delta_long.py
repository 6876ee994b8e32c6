"""The gated delta rule on the GPU where a call has many heads or many tokens: a workgroup of
whole heads, sequences that are taken in pieces, tensors past 2^31 elements; strengths next to
zero; and the operators of a layer one after the other, with their gradients."""
import pytest
import torch

import delta_ref as ref
from gpu_common import need_gpu, say
from linear_ref import f64
from test_gpu_delta import ARGS, BF, F32, _rand, check_backward, check_prefill, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("B,T,H,Hk,lens", [(16, 70, 8, 4, None), (33, 65, 4, 4, [65, 0, 1, 64, 63, 33, -2, 99, 17] * 3 + [65] * 6),
                                            (2, 150, 64, 16, [150, 129])])
def test_prefill_of_many_heads(B, T, H, Hk, dk, lens):
    """From 128 heads of 128 value channels on a workgroup takes a whole head."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("delta prefill of many heads", B, T, H, Hk, dk)
    x, _ = make(B, T, H, Hk, dk, 128, BF, seed=B, lens=lens)
    if lens is not None:
        for b, n in enumerate(lens):
            for t in ("q", "k", "v", "g", "beta"):
                x[t][b, max(n, 0):] = float("nan")
    o, S_T = kda.delta_prefill(*(x[n] for n in ARGS), x["S0"], x["lens"])
    torch.cuda.synchronize()
    if lens is not None:
        for b, n in enumerate(lens):
            assert not o[b, max(n, 0):].any()
            for t in ("q", "k", "v", "g", "beta"):
                x[t][b, max(n, 0):] = 0
    check_prefill(x, o, S_T)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("B,H,dv,dtype", [(4, 24, 32, BF), (16, 8, 128, BF), (4, 24, 32, F32)])
def test_long_sequences_are_the_pieces_one_after_the_other(B, H, dv, dtype, paged):
    """A call whose chunks' operands pass 384 MiB goes window by window with the state between them in
    the workspace: the same bits as a call for each window.  One sequence ends within the first
    window, one has no tokens; with pages, one is skipped."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    chunks, dk = 220, 32
    T = 64 * chunks - 7
    lens = [T, 1000, 0] + [T - 65] * (B - 3)
    x, gen = make(B, T, H, H, dk, dv, dtype, seed=H, lens=lens)
    kw = dict(dtype=torch.int32, device="cuda")
    one = kda.kda_delta_prefill_workspace_bytes(B, 64 * 8, H, H, dk, dv, dtype) // 8     # of a chunk
    n = -(-chunks // ((384 << 20) // one))
    assert n > 1
    step = 64 * -(-chunks // n)
    S, os = x["S0"], []
    for at in range(0, T, step):
        piece = {t: x[t][:, at:at + step].contiguous() for t in ("q", "k", "v", "g", "beta")}
        here = torch.tensor([min(max(l - at, 0), step) for l in lens], **kw)
        o, S = kda.delta_prefill(*piece.values(), x["scale"], S, here)
        os.append(o)
    want = torch.cat(os, 1)
    if not paged:
        o, S_T = kda.delta_prefill(*(x[t] for t in ARGS), x["S0"], x["lens"])
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(S_T, S)
        return
    slots = torch.randperm(B + 5, generator=torch.Generator().manual_seed(1))[:B].int()
    pool = _rand(gen, B + 5, H, dk, dv)
    pool[slots.long().cuda()] = x["S0"]
    want_pool = pool.clone()
    slots[3] = -1
    want[3] = 7.0
    for b in range(B):
        if b != 3:
            want_pool[int(slots[b])] = S[b]
            want[b, max(lens[b], 0):] = 7.0
    o = torch.full_like(x["v"], 7.0)
    ws = torch.empty(kda.kda_delta_prefill_workspace_bytes(B, T, H, H, dk, dv, dtype), dtype=torch.uint8, device="cuda")
    kda.kda_delta_prefill_paged(*(x[t] for t in ARGS), pool, slots.cuda(), slots.cuda(), o, x["lens"], ws)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(pool, want_pool)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strengths_next_to_zero(dtype):
    """Down to the smallest fp32 values, of both signs, and nothing at all in a whole chunk: dbeta
    does not divide by them."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, gen = make(2, 200, 4, 2, 64, 64, dtype, seed=31)
    x["beta"][:, ::5] = torch.tensor([0.0, 1e-30, -1e-25, 2.0 ** -61, 1e-45, -(2.0 ** -60)], device="cuda").repeat(7)[None, :40, None]
    x["beta"][0, 64:128] = 0.0
    x["v"][0, 70] = 1e30                               # not written
    x["dO"], x["dS_T"] = _rand(gen, *x["v"].shape).to(dtype), _rand(gen, *x["S0"].shape)
    o, S_T = kda.delta_prefill(*(x[n] for n in ARGS), x["S0"])
    torch.cuda.synchronize()
    check_prefill(x, o, S_T)
    x["v"][0, 70] = 0.0
    got = kda.delta_backward(*(x[n] for n in ARGS[:5]), x["dO"], x["scale"], x["S0"], x["dS_T"])
    torch.cuda.synchronize()
    check_backward(x, got)
    assert not got["dv"][0, 64:128].any()


def test_single_tokens_of_a_pool_past_32_bits():
    """Slots whose states lie past 2^31 elements of the pool."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, gen = make(3, 1, 8, 8, 128, 128, BF, seed=41, one=True)
    n = (1 << 31) // (8 * 128 * 128) + 40
    pool = torch.empty(n, 8, 128, 128, device="cuda")
    slots = torch.tensor([n - 1, 2, n - 30], dtype=torch.int32, device="cuda")
    pool[slots.long()] = x["S0"]
    o = torch.empty_like(x["v"])
    kda.kda_delta_decode_step_paged(*(x[t] for t in ARGS), pool, slots, o)
    S = x["S0"].clone()
    want = kda.delta_decode_step(*(x[t] for t in ARGS[:5]), S, x["scale"])
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(pool[slots.long()], S)


def test_prefill_past_32_bits():
    """The last sequences of tensors of more than 2^31 elements."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    B, T, H = 66, 8192, 32
    few, _ = make(2, T, H, H, 128, 128, BF, seed=42, state=False)
    big = {n: torch.zeros(B, *few[n].shape[1:], dtype=few[n].dtype, device="cuda") for n in ("q", "k", "v", "g", "beta")}
    for n in big:
        big[n][-2:] = few[n]
    lens = torch.tensor([0] * (B - 2) + [T, T - 3], dtype=torch.int32, device="cuda")
    o, S_T = kda.delta_prefill(*big.values(), few["scale"], lens=lens)
    want, S = kda.delta_prefill(*(few[n] for n in ARGS), lens=lens[-2:])
    torch.cuda.synchronize()
    assert not o[:2].any() and not S_T[:2].any()
    # another split of the work: o off by a rounding, the states by some of fp32
    assert (f64(o[-2:]) - f64(want)).norm() <= 2.0 ** -8 * f64(want).norm()
    assert (f64(S_T[-2:]) - f64(S)).norm() <= 64 * 2.0 ** -24 * f64(S).norm()


def test_block_norm_past_32_bits():
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    D = 4096
    rows = (1 << 31) // D + 9
    r = torch.zeros(rows, D, dtype=BF, device="cuda")
    y = torch.zeros(rows, D, dtype=BF, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    r[-5:], y[-5:] = _rand(gen, 5, D).to(BF), _rand(gen, 5, D).to(BF)
    h, n = kda.block_norm(y, r, norm_y=True, scale=0.5)
    hs, ns = kda.block_norm(y[-5:].clone(), r[-5:].clone(), norm_y=True, scale=0.5)
    torch.cuda.synchronize()
    assert torch.equal(h[-5:], hs) and torch.equal(n[-5:], ns) and not h[:5].any()


# ----------------------------------------------------------------- a layer

def _layer64(p, x, eps):
    """The layer below in 64 bits on the CPU, differentiable: (the stream, the next norm's output)."""
    T, H, dk = x["T"], x["H"], x["dk"]
    n = lambda t: t / torch.sqrt(t.square().mean(-1, keepdim=True) + eps)  # noqa: E731
    a = n(p["r"]) * p["w_in"]
    q, k, v = (a @ p[m] for m in ("Wq", "Wk", "Wv"))
    q, k = n(q.reshape(T, H, dk)) / dk ** 0.5, n(k.reshape(T, H, dk)) / dk ** 0.5
    v, z = v.reshape(T, H, -1), (a @ p["Wz"]).reshape(T, H, -1)
    S = torch.zeros(H, dk, v.shape[-1], dtype=torch.float64)
    out = []
    for t in range(T):
        S = torch.exp(p["g"][t])[:, None, None] * S
        e = v[t] - (k[t][:, :, None] * S).sum(1)
        S = S + k[t][:, :, None] * (p["beta"][t][:, None] * e)[:, None]
        out.append((q[t][:, :, None] * S).sum(1))
    o = torch.stack(out)
    y = n(o) * p["w_o"] * (z * torch.sigmoid(z))
    u = y.reshape(T, -1) @ p["Wo"]
    h = p["r"] + n(u) * p["w_y"]
    return h, n(h) * p["w_n"]


def test_a_layer_of_the_operators():
    """Norm, projections, norm of q and k, the rule over a prompt, its gated norm, the projection
    back, and the norm between blocks; the prompt's last tokens one at a time; and the gradients
    back through all of it, against 64 bits.  Each of the nine steps is off by at most the fp32
    roundings of its longest sum (256 terms, or the T tokens), 2^-24 each, of its norm."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    T, D, H, dk, dv, eps, last = 150, 256, 4, 32, 64, 1e-6, 3
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: _rand(gen, *s)  # noqa: E731
    w = dict(r=rnd(T, D), w_in=1 + 0.1 * rnd(D), Wq=rnd(D, H * dk) / 16, Wk=rnd(D, H * dk) / 16, Wv=rnd(D, H * dv) / 16,
             Wz=rnd(D, H * dv) / 16, Wo=rnd(H * dv, D) / 16, w_o=1 + 0.1 * rnd(dv), w_y=1 + 0.1 * rnd(D), w_n=1 + 0.1 * rnd(D),
             g=-torch.exp2(-6 * torch.rand(T, H, generator=gen, device="cuda")), beta=torch.sigmoid(rnd(T, H)))
    dh, dn = rnd(T, D), rnd(T, D)
    ones = torch.full((dk,), dk ** -0.5, device="cuda")

    # ---- forward: a prompt and its last tokens
    _, a = kda.block_norm(None, w["r"], w_n=w["w_in"], eps=eps)
    q0, k0 = (a @ w["Wq"]).view(1, T, H, dk), (a @ w["Wk"]).view(1, T, H, dk)
    v, z = (a @ w["Wv"]).view(1, T, H, dv), (a @ w["Wz"]).view(1, T, H, dv)
    q, k = kda.qk_norm_rope(q0, k0, w_q=ones, w_k=ones, eps=eps)
    g, beta = w["g"][None].contiguous(), w["beta"][None].contiguous()
    m = T - last
    o, S = kda.delta_prefill(*(t[:, :m].contiguous() for t in (q, k, v, g, beta)))
    tail = [kda.delta_decode_step(*(t[:, i].contiguous() for t in (q, k, v, g, beta)), S) for i in range(m, T)]
    o = torch.cat([o, torch.stack(tail, 1)], 1)
    y = kda.gated_norm(o, z, w["w_o"], act="silu", eps=eps)
    u = y.view(T, H * dv) @ w["Wo"]
    h, n = kda.block_norm(u, w["r"], w_y=w["w_y"], w_n=w["w_n"], norm_y=True, eps=eps)

    # ---- backward
    b = kda.block_norm_backward(u, h, dn, dh, w_y=w["w_y"], w_n=w["w_n"], norm_y=True, eps=eps)
    gn = kda.gated_norm_backward(o, z, w["w_o"], (b["dy"] @ w["Wo"].T).view(1, T, H, dv), act="silu", eps=eps)
    d = kda.delta_backward(q, k, v, g, beta, gn["dx"], want_dS0=False)
    qk = kda.qk_norm_rope_backward(q0, k0, None, None, d["dq"], d["dk"], w_q=ones, w_k=ones, eps=eps)
    rows = lambda t: t.reshape(T, -1)  # noqa: E731
    da = rows(qk["dq"]) @ w["Wq"].T + rows(qk["dk"]) @ w["Wk"].T + rows(d["dv"]) @ w["Wv"].T + rows(gn["dz"]) @ w["Wz"].T
    first = kda.block_norm_backward(None, w["r"], da, b["dr"], w_n=w["w_in"], eps=eps)
    torch.cuda.synchronize()

    p = {name: f64(t).requires_grad_() for name, t in w.items()}
    H64, N64 = _layer64(p, dict(T=T, H=H, dk=dk), eps)
    ((H64 * f64(dh)).sum() + (N64 * f64(dn)).sum()).backward()
    got = dict(r=first["dr"], w_in=first["dw_n"], Wq=a.T @ rows(qk["dq"]), Wk=a.T @ rows(qk["dk"]), Wv=a.T @ rows(d["dv"]),
               Wz=a.T @ rows(gn["dz"]), Wo=rows(y).T @ b["dy"], w_o=gn["dw"], w_y=b["dw_y"], w_n=b["dw_n"], g=d["dg"][0],
               beta=d["dbeta"][0])
    tol = 9 * 256 * 2.0 ** -24
    pairs = [("h", h, H64), ("n", n, N64)] + [(name, t, p[name].grad) for name, t in got.items()]
    for name, x, want in pairs:
        err = float((f64(x) - want.detach()).norm() / want.detach().norm())
        assert err <= tol, (name, err, tol)
