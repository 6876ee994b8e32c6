"""Cases of linear attention with a decay for each head, of draft trees over its states, and of
the queries' and keys' norm with the position rotation: their inputs, their plain forms in torch,
the library's calls, and their definitions in 64 bits.

Shapes: q, k [B, T, Hk, dk], v, o [B, T, H, dv] (Hk divides H: value heads share queries and
keys), g [H] the log-decay of each head, states [B, H, dk, dv] in fp32.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
CHUNK = 128      # tokens a chunk of the plain form


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest call: one short prompt of the fp32 test configuration (latency)
        dict(name="prefill tiny fp32", kind="prefill", B=1, T=64, H=2, Hk=2, dk=32, dv=32,
             dtype="fp32", ragged=False, state=False),
        # one ordinary prompt
        dict(name="prefill mid", kind="prefill", B=1, T=4096, H=32, Hk=32, dk=128, dv=128,
             dtype="bf16", ragged=False, state=False),
        # a padded batch of prompts of odd lengths that continue states; four value heads share
        # each head of queries and keys
        dict(name="prefill ragged shared", kind="prefill", B=5, T=1531, H=16, Hk=4, dk=64, dv=128,
             dtype="bf16", ragged=True, state=True),
        # long prompts of a batch, continued from states
        dict(name="prefill batched", kind="prefill", B=8, T=8192, H=32, Hk=32, dk=128, dv=128,
             dtype="bf16", ragged=False, state=True),
        # a training step's gradients of one sequence
        dict(name="backward mid", kind="backward", B=1, T=4096, H=32, Hk=32, dk=128, dv=128,
             dtype="bf16", ragged=False, state=False),
        # fp32 training on a padded batch with shared heads and gradients of the states
        dict(name="backward ragged fp32", kind="backward", B=3, T=333, H=8, Hk=2, dk=64, dv=64,
             dtype="fp32", ragged=True, state=True),
        # one token of one sequence (latency)
        dict(name="decode one", kind="decode", B=1, H=32, Hk=32, dk=128, dv=128, dtype="bf16"),
        # one token of each sequence of a full serving batch
        dict(name="decode batch", kind="decode", B=256, H=32, Hk=32, dk=128, dv=128,
             dtype="bf16"),
        # a few drafted tokens of two sequences, then the accepted path enters the states
        dict(name="tree small", kind="tree", B=2, T=13, H=32, Hk=8, dk=128, dv=128, dtype="bf16"),
        # full draft trees of a serving batch
        dict(name="tree batch", kind="tree", B=64, T=64, H=32, Hk=32, dk=128, dv=128,
             dtype="bf16"),
        # queries and keys of a prompt: unit rows, rotated over the whole head
        dict(name="norm rope mid", kind="norm_rope", B=1, T=4096, H=32, Hk=32, d=128, rot=128,
             interleaved=False, norm="l2", weights=False, dtype="bf16", far=0),
        # their gradients in training: RMS norm with weights, shared key heads, half of the head
        # rotated in neighbouring pairs, positions deep in a long context
        dict(name="norm rope backward", kind="norm_rope_backward", B=2, T=1001, H=32, Hk=8, d=128,
             rot=64, interleaved=True, norm="rms", weights=True, dtype="bf16", far=1000000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(["prefill", "prefill", "backward", "decode", "tree", "norm_rope",
                       "norm_rope_backward"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    Hk = rng.choice([1, 2, 3, 4, 8, 16, 32])
    H = Hk * rng.choice([1, 1, 2, 4])
    dk, dv = rng.choice([32, 64, 128, 128]), rng.choice([32, 64, 128, 128])
    if H > 32:
        H = Hk = 32
    if kind in ("prefill", "backward"):
        most = 8 * 8192 * 32 // (1 if kind == "prefill" else 16)     # token-heads
        most //= 1 if dtype == "bf16" else 2
        B = _log(rng, 1, 8)
        T = _log(rng, 1, max(1, min(8192 if kind == "prefill" else 4096, most // (B * H))))
        return dict(kind=kind, B=B, T=T, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype,
                    ragged=rng.random() < 0.5, state=rng.random() < 0.5)
    if kind == "decode":
        return dict(kind=kind, B=_log(rng, 1, 256), H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype)
    if kind == "tree":
        return dict(kind=kind, B=_log(rng, 1, 64), T=_log(rng, 1, 64), H=H, Hk=Hk, dk=dk, dv=dv,
                    dtype=dtype)
    d = rng.choice([32, 64, 128])
    B = _log(rng, 1, 16)
    return dict(kind=kind, B=B, T=_log(rng, 1, 8192 // B), H=H, Hk=Hk, d=d,
                rot=2 * rng.randint(1, d // 2), interleaved=rng.random() < 0.5,
                norm=rng.choice(["l2", "rms"]), weights=rng.random() < 0.5, dtype=dtype,
                far=rng.choice([0, 4096, 1000000]))


def work(c):
    kind, es = c["kind"], 2 if c["dtype"] == "bf16" else 4
    if kind.startswith("norm_rope"):
        n = c["B"] * c["T"] * (c["H"] + c["Hk"]) * c["d"]
        extra = c["B"] * c["T"] * 4 + 2 * c["d"] * 4
        back = kind.endswith("backward")
        return dict(bytes=n * es * (3 if back else 2) + extra * (2 if back else 1),
                    flops=n * (12 if back else 7))
    B, H, Hk, dk, dv = (c[x] for x in ("B", "H", "Hk", "dk", "dv"))
    T = c.get("T", 1)
    qk, vo, S = 2 * B * T * Hk * dk * es, 2 * B * T * H * dv * es, B * H * dk * dv * 4
    pair = B * T * H * dk * dv
    if kind == "prefill":
        return dict(bytes=qk + vo + S * (2 if c["state"] else 1), flops=4 * pair)
    if kind == "backward":
        # q, k, v, dO in; dq, dk, dv out; S0 and dS_T in where there are states, dS0 out
        return dict(bytes=2 * qk + vo + vo // 2 + S * (3 if c["state"] else 1), flops=10 * pair)
    if kind == "decode":
        return dict(bytes=qk + vo + 2 * S, flops=4 * pair)
    return dict(bytes=qk + vo + 2 * S + B * (T + 1) * 4,
                flops=2 * pair + 2 * B * H * dk * dv + 2 * B * H * T * (dk + dv))


# ------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _unit(x):
    return x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)


def prepare(c, seed):
    gen, dt = _gen(seed), DTYPES[c["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def randint(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device="cuda")

    B, H, Hk, T = c["B"], c["H"], c["Hk"], c.get("T", 1)
    s = dict(c)
    if c["kind"].startswith("norm_rope"):
        d, rot = c["d"], c["rot"]
        s["q"], s["k"] = randn(B, T, H, d).to(dt), randn(B, T, Hk, d).to(dt)
        s["w_q"] = 1.0 + 0.2 * randn(d) if c["weights"] else None
        s["w_k"] = 1.0 + 0.2 * randn(d) if c["weights"] else None
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda") / rot)
        s["positions"] = (torch.arange(T, device="cuda")[None] + randint(0, c["far"] + 1, B, 1)).to(torch.int32)
        if c["kind"].endswith("backward"):
            s["dy_q"], s["dy_k"] = randn(B, T, H, d).to(dt), randn(B, T, Hk, d).to(dt)
        return s
    dk, dv = c["dk"], c["dv"]
    one = c["kind"] == "decode"
    lead = (B,) if one else (B, T)
    s["q"], s["k"] = (_unit(randn(*lead, Hk, dk)).to(dt) for _ in range(2))
    s["v"] = randn(*lead, H, dv).to(dt)
    # decays from half-lives of a few tokens to a few thousand, one for each head
    s["g"] = -torch.exp2(-12.0 * torch.rand(H, generator=gen, device="cuda"))
    s["scale"] = dk ** -0.5
    with_state = c.get("state", True)
    s["S"] = 0.1 * randn(B, H, dk, dv) if with_state else None
    if c["kind"] in ("prefill", "backward"):
        s["lens"] = randint(0, T + 1, B).to(torch.int32) if c["ragged"] else None
        if c["ragged"]:
            s["lens"][0] = T                                            # padded to the longest
    if c["kind"] == "prefill" and c["ragged"]:
        s["o"] = torch.zeros(B, T, H, dv, dtype=dt, device="cuda")      # rows past the lengths stay
    if c["kind"] == "backward":
        s["dO"] = randn(B, T, H, dv).to(dt)
        s["dS_T"] = randn(B, H, dk, dv) if with_state else None
        if c["ragged"]:
            s["grads"] = tuple(torch.zeros_like(s[n]) for n in "qkv")
    if c["kind"] == "tree":
        # the parent of a node is one of the few nodes before it, or the state (-1); behind the
        # drafted nodes of a sequence there are none (-2)
        t = torch.arange(T, device="cuda")
        back = 1 + (4.0 * torch.rand(B, T, generator=gen, device="cuda")).long()
        parent = torch.clamp(t - back, min=-1)
        count = randint(1, T + 1, B)
        s["parent"] = torch.where(t < count[:, None], parent, -2).to(torch.int32)
        s["accepted"] = (torch.rand(B, generator=gen, device="cuda") * (count + 1)).long().clamp(max=T).sub(1).to(torch.int32)
        s["S_out"] = torch.empty_like(s["S"])
    return s


# ------------------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    plain = dict(prefill=_prefill, backward=_backward, decode=_decode, tree=_tree,
                 norm_rope=_norm_rope, norm_rope_backward=_norm_rope_backward)
    return plain[s["kind"]](s)


def _run_own(s):
    import linear_attention_recurrence_05_amd as kda
    kind = s["kind"]
    if kind == "prefill":
        o, S_T = kda.linear_prefill(s["q"], s["k"], s["v"], s["g"], s["scale"], S0=s["S"],
                                    lens=s["lens"], o=s.get("o"))
        return dict(o=o, S_T=S_T)
    if kind == "backward":
        dq, dk, dv = s.get("grads", (None, None, None))
        return kda.linear_backward(s["q"], s["k"], s["v"], s["g"], s["dO"], s["scale"],
                                   S0=s["S"], dS_T=s["dS_T"], lens=s["lens"], dq=dq, dk=dk, dv=dv)
    if kind == "decode":
        o = kda.linear_decode_step(s["q"], s["k"], s["v"], s["g"], s["S"], s["scale"])
        return dict(o=o, S=s["S"])
    if kind == "tree":
        o = kda.linear_tree(s["q"], s["k"], s["v"], s["g"], s["S"], s["parent"], s["scale"])
        S_out = kda.linear_tree_commit(s["k"], s["v"], s["g"], s["S"], s["parent"], s["accepted"],
                                       S_out=s["S_out"])
        return dict(o=o, S_out=S_out)
    if kind == "norm_rope":
        q, k = kda.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], w_q=s["w_q"],
                                w_k=s["w_k"], norm=s["norm"], eps=EPS,
                                interleaved=s["interleaved"])
        return dict(q=q, k=k)
    return kda.qk_norm_rope_backward(s["q"], s["k"], s["positions"], s["inv_freq"], s["dy_q"],
                                     s["dy_k"], w_q=s["w_q"], w_k=s["w_k"], norm=s["norm"],
                                     eps=EPS, interleaved=s["interleaved"])


# ------------------------------------------------------------------------------------- plain forms

def _heads(x, H):
    """[B, T, h, d] as fp32 [B, H, T, d], a shared head repeated for each that uses it."""
    return x.float().repeat_interleave(H // x.shape[2], dim=2).transpose(1, 2)


def _chunks(x, C):
    """[B, H, T, d] padded with zero tokens and cut: [B, H, N, C, d]."""
    B, H, T, d = x.shape
    N = -(-T // C)
    return torch.nn.functional.pad(x, (0, 0, 0, N * C - T)).reshape(B, H, N, C, d)


def _whole(x, T):
    """[B, H, N, C, d] back to [B, T, H, d]."""
    B, H, N, C, d = x.shape
    return x.reshape(B, H, N * C, d)[:, :, :T].transpose(1, 2)


def _lens(s):
    B, T = s["B"], s["T"]
    if s["lens"] is None:
        return torch.full((B,), T, device="cuda"), torch.ones(B, T, dtype=torch.bool, device="cuda")
    n = s["lens"].long()
    return n, torch.arange(T, device="cuda") < n[:, None]


def _chunk_setup(s):
    g, T, H = s["g"], s["T"], s["H"]
    n, live = _lens(s)
    C = min(CHUNK, T)
    m = live[:, None, :, None]
    q, k, v = (torch.where(m, _heads(s[x], H), 0.0) for x in "qkv")
    i = torch.arange(C, device="cuda")
    gap = (i[:, None] - i).clamp(min=0)
    D = torch.where(i[:, None] >= i, torch.exp(g[:, None, None] * gap), 0.0)[:, None]   # [H, 1, C, C]
    t = torch.arange(T, device="cuda")
    left = (n[:, None] - 1 - t).clamp(min=0)                                             # [B, T]
    to_end = torch.where(live[:, None], torch.exp(g[:, None] * left[:, None]), 0.0)      # [B, H, T]
    last = torch.exp(g * n[:, None])[:, :, None, None]                                   # [B, H, 1, 1]
    grow = torch.exp(g[:, None] * (i + 1))[:, None, :, None]                             # [H, 1, C, 1]
    return q, k, v, n, live, C, D, to_end, last, grow


def _starts(s, k, v, C):
    """The state before every chunk, [B, H, N, dk, dv]."""
    g, S0 = s["g"], s["S"]
    kc, vc = _chunks(k, C), _chunks(v, C)
    B, H, N, _, dk = kc.shape
    i = torch.arange(C, device="cuda")
    w = torch.exp(g[:, None] * (C - 1 - i))[:, None, :, None]
    U = (kc * w).transpose(-1, -2) @ vc
    m = torch.arange(N, device="cuda")
    gap = C * (m[:, None] - 1 - m).clamp(min=0)
    L = torch.where(m[:, None] > m, torch.exp(g[:, None, None] * gap), 0.0)
    S = (L @ U.reshape(B, H, N, -1)).reshape(U.shape)
    if S0 is not None:
        S = S + torch.exp(g[:, None] * (C * m))[:, :, None, None] * S0[:, :, None]
    return S


def _prefill(s):
    q, k, v, n, live, C, D, to_end, last, grow = _chunk_setup(s)
    qc, kc, vc = _chunks(q, C), _chunks(k, C), _chunks(v, C)
    o = ((qc @ kc.transpose(-1, -2)) * D) @ vc + grow * (qc @ _starts(s, k, v, C))
    o = _whole(o * s["scale"], s["T"]).to(s["v"].dtype)
    S_T = (k * to_end[..., None]).transpose(-1, -2) @ v
    if s["S"] is not None:
        S_T = S_T + last * s["S"]
    return dict(o=o.contiguous(), S_T=S_T)


def _shared(x, Hk, dt):
    """[B, T, H, d]: the gradients of the heads that share one, summed: [B, T, Hk, d]."""
    B, T, H, d = x.shape
    return x.reshape(B, T, Hk, H // Hk, d).sum(3).to(dt)


def _backward(s):
    g, scale, T, Hk, dt = s["g"], s["scale"], s["T"], s["Hk"], s["q"].dtype
    q, k, v, n, live, C, D, to_end, last, grow = _chunk_setup(s)
    dO = torch.where(live[:, None, :, None], _heads(s["dO"], s["H"]), 0.0)
    qc, kc, vc, dc = (_chunks(x, C) for x in (q, k, v, dO))
    N = qc.shape[2]
    PO = (dc @ vc.transpose(-1, -2)) * D
    PQ = (qc @ kc.transpose(-1, -2)) * D
    dq = PO @ kc + grow * (dc @ _starts(s, k, v, C).transpose(-1, -2))
    # what reaches the end of every chunk from the tokens behind it
    Q = (qc * grow).transpose(-1, -2) @ dc
    m = torch.arange(N, device="cuda")
    gap = C * (m - 1 - m[:, None]).clamp(min=0)
    L = torch.where(m > m[:, None], torch.exp(g[:, None, None] * gap), 0.0)
    R = (L @ Q.reshape(*Q.shape[:3], -1)).reshape(Q.shape)
    i = torch.arange(C, device="cuda")
    back = torch.exp(g[:, None] * (C - 1 - i))[:, None, :, None]
    dk = PO.transpose(-1, -2) @ qc + back * (vc @ R.transpose(-1, -2))
    dv = PQ.transpose(-1, -2) @ dc + back * (kc @ R)
    dq, dk, dv = (_whole(x * scale, T) for x in (dq, dk, dv))
    # every token's way back to the state before the first
    a_i = torch.exp(g[:, None] * (torch.arange(T, device="cuda") + 1))[:, :, None]
    dS0 = scale * ((q * a_i).transpose(-1, -2) @ dO)
    if s["dS_T"] is not None:
        w = to_end[..., None]
        dk = dk + (w * (v @ s["dS_T"].transpose(-1, -2))).transpose(1, 2)
        dv = dv + (w * (k @ s["dS_T"])).transpose(1, 2)
        dS0 = dS0 + last * s["dS_T"]
    return dict(dq=_shared(dq, Hk, dt), dk=_shared(dk, Hk, dt), dv=dv.to(dt).contiguous(), dS0=dS0)


def _decode(s):
    H, S = s["H"], s["S"]
    q, k = (s[x].float().repeat_interleave(H // s["Hk"], dim=1) for x in "qk")
    S.mul_(torch.exp(s["g"])[:, None, None])
    S.add_(k[..., :, None] * s["v"].float()[..., None, :])
    o = s["scale"] * (S * q[..., :, None]).sum(2)
    return dict(o=o.to(s["v"].dtype), S=S)


def _tree(s):
    g, T, S, H = s["g"], s["T"], s["S"], s["H"]
    q, k, v = (_heads(s[x], H) for x in "qkv")
    parent = s["parent"].long()
    B = parent.shape[0]
    t = torch.arange(T, device="cuda")
    # reach[b, i, j]: j is i or above it; doubled until the longest path is covered
    step = ((parent[:, :, None] == t) & (parent[:, :, None] >= 0)).float()
    reach = step + torch.eye(T, device="cuda")
    for _ in range((T - 1).bit_length()):
        reach = torch.clamp(reach @ reach, max=1.0)
    top = ((parent == -1).float()[:, None, :] * reach).sum(2) > 0      # hangs on the state
    depth = reach.sum(2)
    gap = (depth[:, :, None] - depth[:, None, :]).clamp(min=0)[:, None]
    D = torch.where((reach > 0)[:, None], torch.exp(g[:, None, None] * gap), 0.0)
    o = ((q @ k.transpose(-1, -2)) * D) @ v
    o = o + torch.exp(g[:, None] * depth[:, None])[..., None] * (q @ S)
    o = torch.where(top[:, None, :, None], o * s["scale"], 0.0).transpose(1, 2)
    # the accepted node's row of D weighs its path; with none accepted the state stays
    x = s["accepted"].long()
    some = (x >= 0)[:, None, None]
    row = D[torch.arange(B, device="cuda"), :, x.clamp(min=0)]
    n = torch.where(x >= 0, depth[torch.arange(B, device="cuda"), x.clamp(min=0)], 0.0)
    w = torch.where(some, row, 0.0)[..., None]
    new = torch.exp(g * n[:, None])[:, :, None, None] * S + (k * w).transpose(-1, -2) @ v
    s["S_out"].copy_(new)
    return dict(o=o.to(s["v"].dtype).contiguous(), S_out=s["S_out"])


def _angles(s):
    """cos and sin [B, T, 1, rot / 2]; the angles of far positions need 64 bits."""
    a = s["positions"].double()[..., None, None] * s["inv_freq"].double()
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin, rot, interleaved):
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _norm_rope(s):
    cos, sin = _angles(s)
    c = 1.0 if s["norm"] == "l2" else 1.0 / s["d"]

    def one(x, w):
        x = x.float()
        y = x * torch.rsqrt(c * (x * x).sum(-1, keepdim=True) + EPS)
        return _rotate(y if w is None else y * w, cos, sin, s["rot"], s["interleaved"])

    dt = s["q"].dtype
    return dict(q=one(s["q"], s["w_q"]).to(dt), k=one(s["k"], s["w_k"]).to(dt))


def _norm_rope_backward(s):
    cos, sin = _angles(s)
    c = 1.0 if s["norm"] == "l2" else 1.0 / s["d"]

    def one(x, dy, w):
        x = x.float()
        r = torch.rsqrt(c * (x * x).sum(-1, keepdim=True) + EPS)
        du = _rotate(dy.float(), cos, -sin, s["rot"], s["interleaved"])
        dn = du if w is None else du * w
        dx = r * dn - c * r * r * r * x * (x * dn).sum(-1, keepdim=True)
        return dx, None if w is None else (du * x * r).sum((0, 1, 2))

    dt = s["q"].dtype
    dq, dw_q = one(s["q"], s["dy_q"], s["w_q"])
    dk, dw_k = one(s["k"], s["dy_k"], s["w_k"])
    return dict(dq=dq.to(dt), dk=dk.to(dt), dw_q=dw_q, dw_k=dw_k)


# ------------------------------------------------------------------------------------- in 64 bits

def exact(c, seed):
    """The definitions: the recurrence token by token, the gradients as sums over pairs of
    tokens, the tree node by node."""
    s = prepare(c, seed)
    fn = dict(prefill=_exact_prefill, backward=_exact_backward, decode=_exact_decode,
              tree=_exact_tree, norm_rope=_exact_norm, norm_rope_backward=_exact_norm_backward)
    return fn[c["kind"]](s)


def _state64(s):
    if s["S"] is None:
        return torch.zeros(s["B"], s["H"], s["dk"], s["dv"], dtype=torch.float64, device="cuda")
    return s["S"].double()


def _exact_prefill(s):
    H, G = s["H"], s["H"] // s["Hk"]
    a = torch.exp(s["g"].double())[None, :, None, None]
    S, o = _state64(s), torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    of = torch.arange(H, device="cuda") // G
    for t in range(s["T"]):
        q, k = s["q"][:, t].double()[:, of], s["k"][:, t].double()[:, of]
        new = a * S + k[..., None] * s["v"][:, t].double()[:, :, None]
        y = s["scale"] * (q[:, :, None] @ new)[:, :, 0]
        if s["lens"] is not None:
            on = (t < s["lens"])[:, None, None]
            y, new = torch.where(on, y, 0.0), torch.where(on[..., None], new, S)
        S, o[:, t] = new, y
    return dict(o=o, S_T=S)


def _exact_backward(s):
    B, T, H, G = s["B"], s["T"], s["H"], s["H"] // s["Hk"]
    z = dict(dtype=torch.float64, device="cuda")
    dq, dk = (torch.zeros(s["q"].shape, **z) for _ in range(2))
    dv, dS0 = torch.zeros(s["v"].shape, **z), torch.zeros(B, H, s["dk"], s["dv"], **z)
    lens = [T] * B if s["lens"] is None else s["lens"].tolist()
    S, end = _state64(s), torch.zeros_like(_state64(s)) if s["dS_T"] is None else s["dS_T"].double()
    for b in range(B):
        n = lens[b]
        t = torch.arange(n, **z)
        for h in range(H):
            g = s["g"][h].double()
            q, k = s["q"][b, :n, h // G].double(), s["k"][b, :n, h // G].double()
            v, dO = s["v"][b, :n, h].double(), s["dO"][b, :n, h].double()
            W = torch.tril(torch.exp(g * (t[:, None] - t).clamp(min=0))) * s["scale"]
            X = W * (dO @ v.T)
            first, behind = torch.exp(g * (t + 1))[:, None], torch.exp(g * (n - 1 - t))[:, None]
            dq[b, :n, h // G] += X @ k + s["scale"] * first * (dO @ S[b, h].T)
            dk[b, :n, h // G] += X.T @ q + behind * (v @ end[b, h].T)
            dv[b, :n, h] = (W * (q @ k.T)).T @ dO + behind * (k @ end[b, h])
            dS0[b, h] = torch.exp(g * n) * end[b, h] + s["scale"] * (first * q).T @ dO
    return dict(dq=dq, dk=dk, dv=dv, dS0=dS0)


def _exact_decode(s):
    of = torch.arange(s["H"], device="cuda") // (s["H"] // s["Hk"])
    a = torch.exp(s["g"].double())[None, :, None, None]
    S = a * s["S"].double() + s["k"].double()[:, of][..., None] * s["v"].double()[:, :, None]
    return dict(o=s["scale"] * (s["q"].double()[:, of][:, :, None] @ S)[:, :, 0], S=S)


def _exact_tree(s):
    B, T, G = s["B"], s["T"], s["H"] // s["Hk"]
    of = torch.arange(s["H"], device="cuda") // G
    a = torch.exp(s["g"].double())[:, None, None]
    o, S_out = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda"), s["S"].double()
    parent, accepted = s["parent"].tolist(), s["accepted"].tolist()
    for b in range(B):
        root = s["S"][b].double()
        states = {-1: root}
        q, k, v = s["q"][b].double()[:, of], s["k"][b].double()[:, of], s["v"][b].double()
        for t in range(T):
            if parent[b][t] in states:                                  # -2 never is
                states[t] = a * states[parent[b][t]] + k[t][..., None] * v[t][:, None]
                o[b, t] = s["scale"] * (q[t][:, None] @ states[t])[:, 0]
        S_out[b] = states[accepted[b]]
    return dict(o=o, S_out=S_out)


def _turned(s, x, sign):
    """Pairs as complex numbers, turned by sign times the angle."""
    rot, lead = s["rot"], x.shape[:-1]
    a = sign * s["positions"].double()[:, :, None, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(a), a)
    head, rest = x[..., :rot], x[..., rot:]
    pairs = head.reshape(*lead, rot // 2, 2) if s["interleaved"] else head.reshape(*lead, 2, rot // 2).transpose(-1, -2)
    got = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    got = got if s["interleaved"] else got.transpose(-1, -2)
    return torch.cat([got.reshape(*lead, rot), rest], -1)


def _length64(s, x):
    mean = x.square().sum(-1, keepdim=True) / (1 if s["norm"] == "l2" else s["d"])
    return torch.sqrt(mean + EPS)


def _exact_norm(s):
    out = {}
    for n in "qk":
        x, w = s[n].double(), s["w_" + n]
        y = x / _length64(s, x)
        out[n] = _turned(s, y if w is None else y * w.double(), 1.0)
    return out


def _exact_norm_backward(s):
    out = {}
    for n in "qk":
        x, w = s[n].double(), s["w_" + n]
        size = _length64(s, x)
        unit, du = x / size, _turned(s, s["dy_" + n].double(), -1.0)
        dn = du if w is None else du * w.double()
        c = 1.0 if s["norm"] == "l2" else 1.0 / s["d"]
        out["d" + n] = (dn - c * unit * (unit * dn).sum(-1, keepdim=True)) / size
        out["dw_" + n] = None if w is None else (du * unit).flatten(0, 2).sum(0)
    return out
