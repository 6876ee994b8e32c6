"""The gated delta rule on the GPU against its 64-bit definition: prefill, gradients, single
tokens, paged states."""
import pytest
import torch

import delta_ref as ref
from gpu_common import need_gpu, say
from linear_ref import lengths

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ARGS = ("q", "k", "v", "g", "beta", "scale")


def _rand(gen, *s):
    return torch.randn(*s, generator=gen, device="cuda")


def make(B, T, H, Hk, dk, dv, dtype, seed=0, state=True, lens=None, one=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    unit = lambda x: x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)  # noqa: E731
    lead = (B,) if one else (B, T)
    rate = torch.exp2(-9.0 * torch.rand(H, generator=gen, device="cuda"))
    x = dict(q=unit(_rand(gen, *lead, Hk, dk)).to(dtype), k=unit(_rand(gen, *lead, Hk, dk)).to(dtype),
             v=_rand(gen, *lead, H, dv).to(dtype), g=-rate * _rand(gen, *lead, H).abs(),
             beta=torch.sigmoid(_rand(gen, *lead, H)), scale=dk ** -0.5,
             S0=_rand(gen, B, H, dk, dv) if state else None,
             lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"))
    return x, gen


def terms(*sizes):
    """fp32 sums of that many terms, and decays good to a few 2^-24."""
    return sum(sizes) + 256


def check_prefill(x, o, S_T):
    """bf16: the state is rounded to bf16 once on its way into o, the pairs' weights and what a
    token writes once each.  S_T: fp32 throughout."""
    want = ref.prefill(*(x[n] for n in ARGS), x["S0"], x["lens"])
    n = terms(x["v"].shape[1], x["q"].shape[-1])
    ref.check("o", o, want["o"], want["o_mag"], want["o_sum"], 2 if x["q"].dtype == BF else 0, n)
    if S_T is not None:
        ref.check("S_T", S_T, want["S_T"], None, want["S_sum"], 0, n)


def check_backward(x, got):
    """bf16: as in check_prefill, on three operands of a part of dk; dv, dg, dbeta and dS0 are
    fp32 sums throughout."""
    want, mag, sums = ref.backward(*(x[n] for n in ARGS), x["dO"], x["S0"], x["dS_T"], x["lens"])
    n = terms(2 * x["v"].shape[1], x["q"].shape[-1], x["v"].shape[-1])
    for name in want:
        if got[name] is not None:
            less = x["q"].dtype == BF and name in ("dq", "dk")
            ref.check(name, got[name], want[name], mag[name], sums[name], 3 if less else 0, n)


SIZES = [  # B, T, H, Hk, dk, dv
    (1, 1, 1, 1, 32, 32), (2, 2, 2, 1, 32, 64), (1, 31, 2, 2, 64, 32), (1, 32, 2, 2, 64, 64),
    (2, 33, 4, 2, 128, 128), (3, 65, 3, 1, 128, 32), (1, 127, 2, 2, 32, 128), (2, 300, 6, 3, 64, 128),
    (1, 515, 2, 2, 128, 64), (1, 1100, 1, 1, 128, 128),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", SIZES)
def test_prefill(size, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("delta prefill", size, dtype)
    x, _ = make(*size, dtype, seed=size[1], state=size[1] % 2 == 1)
    o, S_T = kda.delta_prefill(*(x[n] for n in ARGS), x["S0"])
    torch.cuda.synchronize()
    check_prefill(x, o, S_T)


def _hide(x, names, T):
    """NaN behind the lengths, in place; returns the same tensors with zeros there."""
    clean = {n: x[n].clone() for n in names}
    for b, n in enumerate(lengths(x["lens"], x["v"].shape[0], T)):
        for t in names:
            x[t][b, n:] = float("nan")
            clean[t][b, n:] = 0
    return clean


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_lengths_leave_the_rest_alone(dtype):
    """Odd lengths, 0, 1, and values outside [0, T]; rows past them hold NaN and are neither read
    nor written."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    lens = [0, 1, 150, 97, -3, 999, 32, 33]
    B, T = len(lens), 150
    x, _ = make(B, T, 4, 2, 64, 128, dtype, seed=5, lens=lens)
    clean = _hide(x, ("q", "k", "v", "g", "beta"), T)
    o = torch.full((B, T, 4, 128), 7.0, dtype=dtype, device="cuda")
    _, S_T = kda.delta_prefill(*(x[n] for n in ARGS), x["S0"], x["lens"], o=o)
    torch.cuda.synchronize()
    for b, n in enumerate(lengths(lens, B, T)):
        assert (o[b, n:] == 7.0).all()
        o[b, n:] = 0
    check_prefill({**x, **clean}, o, S_T)
    assert torch.equal(S_T[0], x["S0"][0]) and torch.equal(S_T[4], x["S0"][4])
    o2, _ = kda.delta_prefill(*(x[n] for n in ARGS), x["S0"], x["lens"])
    assert torch.equal(o2, o)                       # an allocated o is zero there


def extremes(x):
    """Heads without a decay, with total ones (also -infinity) at some tokens or all, a fast and a
    slow one; heads that write nothing, everything, more than everything."""
    g, beta = x["g"], x["beta"]
    g[:, :, 0] = 0.0
    g[:, :, 1] = float("-inf")
    g[:, ::7, 2] = float("-inf")
    g[:, 3::40, 3] = -1e30
    g[:, :, 4] = -30.0
    g[:, :, 5] = -1e-6
    g[:, 20::50, 5] = -2000.0
    beta[:, :, 0] = 0.0
    beta[:, :, 2] = 1.0
    beta[:, :, 3] = 1.9
    beta[:, 5::9, 5] = 0.0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decays_and_strengths_at_their_ends(dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, gen = make(1, 130, 6, 6, 64, 64, dtype, seed=6)
    extremes(x)
    o, S_T = kda.delta_prefill(*(x[n] for n in ARGS), x["S0"])
    torch.cuda.synchronize()
    check_prefill(x, o, S_T)
    x["dO"], x["dS_T"] = _rand(gen, *x["v"].shape).to(dtype), _rand(gen, *x["S0"].shape)
    got = kda.delta_backward(*(x[n] for n in ARGS[:5]), x["dO"], x["scale"], x["S0"], x["dS_T"])
    torch.cuda.synchronize()
    check_backward(x, got)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_same_key_again_and_again(dtype):
    """Keys that repeat make the pairs of a chunk as large as they get: the triangular system's
    entries are near beta throughout."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, gen = make(2, 100, 2, 1, 128, 64, dtype, seed=7)
    x["k"][:] = x["k"][:, :1]
    x["g"] *= 1e-3
    x["beta"][:, :, 0] = 1.0
    x["beta"][:, :, 1] = 1.8
    x["dO"], x["dS_T"] = _rand(gen, *x["v"].shape).to(dtype), _rand(gen, *x["S0"].shape)
    o, S_T = kda.delta_prefill(*(x[n] for n in ARGS), x["S0"])
    got = kda.delta_backward(*(x[n] for n in ARGS[:5]), x["dO"], x["scale"], x["S0"], x["dS_T"])
    torch.cuda.synchronize()
    check_prefill(x, o, S_T)
    check_backward(x, got)


def test_prefill_in_place_state_and_continuation():
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, _ = make(2, 90, 2, 2, 128, 128, F32, seed=7)
    S = x["S0"].clone()
    o = torch.empty_like(x["v"])
    for lo, hi in ((0, 37), (37, 38), (38, 90)):
        part = [x[n][:, lo:hi].contiguous() for n in ("q", "k", "v", "g", "beta")]
        po = torch.empty_like(part[2])
        ws = torch.empty(max(1, kda.kda_delta_prefill_workspace_bytes(2, hi - lo, 2, 2, 128, 128, F32)),
                         dtype=torch.uint8, device="cuda")
        kda.kda_delta_prefill(*part, x["scale"], S, po, S, workspace=ws)
        o[:, lo:hi] = po
    torch.cuda.synchronize()
    check_prefill(x, o, S)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_in_place_state_of_long_sequences(dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, _ = make(3, 2100, 2, 1, 64, 128, dtype, seed=17, lens=[2100, 700, 31])
    args = [x[n] for n in ARGS]
    o, S_T = kda.delta_prefill(*args, x["S0"], x["lens"])
    ws = torch.empty(max(1, kda.kda_delta_prefill_workspace_bytes(3, 2100, 2, 1, 64, 128, dtype)), dtype=torch.uint8,
                     device="cuda")
    for _ in range(5):
        S, o2 = x["S0"].clone(), torch.zeros_like(o)
        kda.kda_delta_prefill(*args, S, o2, S, x["lens"], ws)
        torch.cuda.synchronize()
        assert torch.equal(S, S_T) and torch.equal(o2, o)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", SIZES[:-2] + [(1, 410, 2, 1, 128, 128)])
def test_backward(size, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("delta backward", size, dtype)
    state = size[1] % 2 == 0
    x, gen = make(*size, dtype, seed=100 + size[1], state=state)
    x["dO"] = _rand(gen, *x["v"].shape).to(dtype)
    x["dS_T"] = _rand(gen, size[0], size[2], size[4], size[5]) if state else None
    got = kda.delta_backward(*(x[n] for n in ARGS[:5]), x["dO"], x["scale"], x["S0"], x["dS_T"])
    torch.cuda.synchronize()
    check_backward(x, got)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hk", [4, 1])
def test_backward_lengths_leave_the_rest_alone(dtype, Hk):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    lens = [0, 1, 101, 64, -1, 500, 33]
    B, T = len(lens), 101
    x, gen = make(B, T, 4, Hk, 64, 32, dtype, seed=8, lens=lens)
    x["dO"], x["dS_T"] = _rand(gen, *x["v"].shape).to(dtype), _rand(gen, B, 4, 64, 32)
    clean = _hide(x, ("q", "k", "v", "dO", "g", "beta"), T)
    out = {n: torch.full_like(x[n[1:]], 7.0) for n in ("dq", "dk", "dv", "dg", "dbeta")}
    got = kda.delta_backward(*(x[n] for n in ARGS[:5]), x["dO"], x["scale"], x["S0"], x["dS_T"], x["lens"], **out)
    torch.cuda.synchronize()
    for b, n in enumerate(lengths(lens, B, T)):
        for t in out.values():
            assert (t[b, n:] == 7.0).all()
            t[b, n:] = 0
    check_backward({**x, **clean}, got)
    assert torch.equal(got["dS0"][0], x["dS_T"][0])


def test_backward_against_differences_of_the_definition():
    """Central differences of the 64-bit definition (width 1e-6 of inputs near 1: good to 1e-9)
    along a random direction, against the gradients' sum along it, each gradient within its
    fp32 sums' tolerance."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, gen = make(2, 75, 4, 2, 64, 32, F32, seed=9)
    x["dO"], x["dS_T"] = _rand(gen, *x["v"].shape), _rand(gen, 2, 4, 64, 32)
    got = kda.delta_backward(*(x[n] for n in ARGS[:5]), x["dO"], x["scale"], x["S0"], x["dS_T"])
    torch.cuda.synchronize()
    _, _, sums = ref.backward(*(x[n] for n in ARGS), x["dO"], x["S0"], x["dS_T"])

    def loss(y):
        out = ref.prefill(*(y[n] for n in ARGS), y["S0"])
        return float((out["o"] * ref.f64(x["dO"])).sum() + (out["S_T"] * ref.f64(x["dS_T"])).sum())

    n = terms(2 * 75, 64, 32)
    for name in ("q", "k", "v", "g", "beta", "S0"):
        way = ref.f64(_rand(gen, *x[name].shape))
        up, down = (loss({**x, name: ref.f64(x[name]) + s * way}) for s in (1e-6, -1e-6))
        d = "d" + name
        want = float((ref.f64(got[d]) * way).sum())
        tol = float(((2.0 ** -24 * ref.f64(got[d]).abs() + n * 2.0 ** -24 * sums[d]) * way.abs()).sum())
        assert abs((up - down) / 2e-6 - want) < tol + 1e-6 * max(abs(want), 1.0), (name, up, down, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [(1, 1, 1, 32, 32), (3, 2, 1, 64, 128), (2, 4, 4, 128, 128), (5, 3, 3, 128, 32),
                                  (2, 6, 2, 32, 64), (2, 2, 2, 32, 128), (40, 32, 32, 128, 128)])
def test_decode(size, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    B, H, Hk, dk, dv = size
    x, _ = make(B, 1, H, Hk, dk, dv, dtype, seed=B, one=True)
    x["g"][0, 0] = float("-inf")
    S = x["S0"].clone()
    o = kda.delta_decode_step(*(x[n] for n in ARGS[:5]), S, x["scale"])
    torch.cuda.synchronize()
    want = ref.decode(*(x[n] for n in ARGS), x["S0"])
    ref.check("o", o, want["o"], None, want["o_sum"], 0, terms(dk))
    ref.check("S", S, want["S_T"], None, want["S_sum"], 0, terms(dk))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_single_tokens_continue_a_prefill(dtype):
    """A prompt by prefill and then its last tokens one by one: the states and outputs of the
    whole."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, _ = make(2, 60, 4, 2, 64, 128, dtype, seed=11)
    cut = 52
    head = [x[n][:, :cut].contiguous() for n in ARGS[:5]]
    o, S = kda.delta_prefill(*head, x["scale"], x["S0"])
    rest = [kda.delta_decode_step(*(x[n][:, t].contiguous() for n in ARGS[:5]), S, x["scale"]) for t in range(cut, 60)]
    torch.cuda.synchronize()
    check_prefill(x, torch.cat([o, torch.stack(rest, 1)], 1), S)


# ----------------------------------------------------------------- paged states

@pytest.mark.parametrize("dtype", [BF, F32])
def test_paged_states(dtype):
    """Slots in any order, states kept and skipped sequences; the same sums as the dense call."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    B, T, H, Hk, dk, dv = 5, 70, 4, 2, 64, 64
    x, gen = make(B, T, H, Hk, dk, dv, dtype, seed=12, lens=[70, 33, 0, 64, 1])
    pool = _rand(gen, 9, H, dk, dv)
    i32 = dict(dtype=torch.int32, device="cuda")
    s_in, s_out = torch.tensor([7, 2, 4, -1, 0], **i32), torch.tensor([7, 3, 5, 6, 9], **i32)
    for tables in ((s_in, s_out), (None, s_out), (s_in, None)):
        p = pool.clone()
        o = torch.full_like(x["v"], 7.0)
        ws = torch.empty(max(1, kda.kda_delta_prefill_workspace_bytes(B, T, H, Hk, dk, dv, dtype)), dtype=torch.uint8, device="cuda")
        kda.kda_delta_prefill_paged(*(x[n] for n in ARGS), p, *tables, o, x["lens"], ws)
        S0 = torch.stack([pool[s] if 0 <= s < 9 else pool[0] for s in (tables[0] if tables[0] is not None else s_out).tolist()])
        S0 = S0 if tables[0] is not None else None
        od, Sd = kda.delta_prefill(*(x[n] for n in ARGS), S0, x["lens"])
        torch.cuda.synchronize()
        want, wo = pool.clone(), torch.full_like(o, 7.0)
        for b, n in enumerate(lengths(x["lens"], B, T)):
            if all(t is None or 0 <= int(t[b]) < 9 for t in tables):
                wo[b, :n] = od[b, :n]
                if tables[1] is not None:
                    want[int(tables[1][b])] = Sd[b]
        assert torch.equal(o, wo) and torch.equal(p, want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_paged_decode(dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, gen = make(4, 1, 6, 3, 128, 64, dtype, seed=13, one=True)
    pool = _rand(gen, 6, 6, 128, 64)
    slots = torch.tensor([5, -1, 0, 6], dtype=torch.int32, device="cuda")
    p, o = pool.clone(), torch.full_like(x["v"], 7.0)
    kda.kda_delta_decode_step_paged(*(x[n] for n in ARGS), p, slots, o)
    S = torch.stack([pool[5], pool[1], pool[0], pool[1]])
    od = kda.delta_decode_step(*(x[n] for n in ARGS[:5]), S, x["scale"])
    torch.cuda.synchronize()
    want, wo = pool.clone(), torch.full_like(o, 7.0)
    want[5], want[0], wo[0], wo[2] = S[0], S[2], od[0], od[2]
    assert torch.equal(p, want) and torch.equal(o, wo)


# ----------------------------------------------------------------- ways to call

@pytest.mark.parametrize("dtype", [BF, F32])
def test_calls_on_a_given_stream(dtype):
    """stream= as a torch stream and as its handle, with another one current."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, gen = make(2, 700, 4, 2, 64, 64, dtype, seed=20)
    dO = _rand(gen, *x["v"].shape).to(dtype)
    args = [x[n] for n in ARGS[:5]]
    want = [*kda.delta_prefill(*args, x["scale"], x["S0"]), *kda.delta_backward(*args, dO, x["scale"], x["S0"]).values()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = [*kda.delta_prefill(*args, x["scale"], x["S0"], stream=stream),
               *kda.delta_backward(*args, dO, x["scale"], x["S0"], stream=stream).values()]
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_two_captured_graphs_share_a_workspace(dtype):
    """Prefill, gradients and a decode step in one graph, and the prefill and gradients of other
    inputs in another, on one workspace; replayed in turn, with eager work between, each gives
    the eager results."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    B, T, H, Hk, d = 2, 333, 4, 2, 64
    ws = torch.empty(max(1, kda.kda_delta_prefill_workspace_bytes(B, T, H, Hk, d, d, dtype),
                         kda.kda_delta_backward_workspace_bytes(B, T, H, Hk, d, d, dtype)), dtype=torch.uint8, device="cuda")

    def plan(seed):
        x, gen = make(B, T, H, Hk, d, d, dtype, seed=seed, lens=[T, 217])
        y, _ = make(B, 1, H, Hk, d, d, dtype, seed=seed + 1, one=True)
        dO, z = _rand(gen, *x["v"].shape).to(dtype), torch.zeros_like
        out = dict(o=z(x["v"]), S=z(x["S0"]), dq=z(x["q"]), dk=z(x["k"]), dv=z(x["v"]), dg=z(x["g"]), dbeta=z(x["beta"]),
                   dS0=z(x["S0"]), o1=z(y["v"]))

        def run():
            kda.kda_delta_prefill(*(x[n] for n in ARGS), x["S0"], out["o"], out["S"], x["lens"], ws)
            kda.kda_delta_backward(*(x[n] for n in ARGS), x["S0"], dO, None, out["dq"], out["dk"], out["dv"], out["dg"],
                                   out["dbeta"], out["dS0"], x["lens"], ws)
            kda.kda_delta_decode_step(*(y[n] for n in ARGS), out["S"], out["o1"])
        return run, out

    plans = [plan(30), plan(40)]
    eager = []
    for run, out in plans:
        run()
        torch.cuda.synchronize()
        eager.append({n: t.clone() for n, t in out.items()})
    graphs = []
    for run, out in plans:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for _ in range(4):
        for g, (run, out), want in zip(graphs, plans, eager):
            for t in out.values():
                t.fill_(7.0)
            for n in ("o", "dq", "dk", "dv", "dg", "dbeta"):
                out[n][1, 217:] = 0
            g.replay()
            torch.cuda.synchronize()
            for n, t in out.items():
                assert torch.equal(t, want[n]), n
            torch.ones(1000, device="cuda").sum().item()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_same_call_gives_the_same_bits(dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, gen = make(2, 1000, 8, 2, 128, 128, dtype, seed=21, lens=[1000, 421])
    dO = _rand(gen, *x["v"].shape).to(dtype)
    args = [x[n] for n in ARGS[:5]]

    def once():
        return [*kda.delta_prefill(*args, x["scale"], x["S0"], x["lens"]),
                *kda.delta_backward(*args, dO, x["scale"], x["S0"], None, x["lens"]).values()]

    want = once()
    for _ in range(3):
        got = once()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# ----------------------------------------------------------------- long sequences

def test_long_slow_decays_keep_their_factor():
    """20,000 tokens at decays near 1, keys of length 1 that write little: the state's error stays
    that of fp32 sums.  Each of 625 chunks rounds the state by at most 2^-24 of itself, at random:
    about sqrt(625) 2^-25 = 7.5e-7 of its norm, to which the weights add a few 2^-24; 4e-6 leaves
    a factor of four.  Chunk factors rounded once would add up to 625 2^-25 = 1.9e-5."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, _ = make(1, 20000, 4, 4, 32, 32, F32, seed=18)
    x["g"] = torch.tensor([-1e-6, -3.1e-5, -1.7e-4, 0.0], device="cuda").expand(1, 20000, 4).contiguous()
    x["beta"] *= 1e-3
    _, S_T = kda.delta_prefill(*(x[n] for n in ARGS), x["S0"])
    torch.cuda.synchronize()
    a = torch.exp(x["g"][0, 0].double())[:, None, None]
    S = x["S0"][0].double()
    for t in range(20000):
        k = x["k"][0, t].double()[:, :, None]
        S = a * S
        S = S + k * (x["beta"][0, t].double()[:, None] * (x["v"][0, t].double() - (k * S).sum(1)))[:, None]
    err = torch.linalg.vector_norm(S_T[0].double() - S, dim=(1, 2)) / torch.linalg.vector_norm(S, dim=(1, 2))
    assert (err < 4e-6).all(), err
