"""Linear attention with a decay for each head on the GPU against its 64-bit
definition: prefill, gradients, single tokens, draft trees, paged states."""
import pytest
import torch

import linear_ref as ref
from gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _rand(gen, *s):
    return torch.randn(*s, generator=gen, device="cuda")


def make(B, T, H, Hk, dk, dv, dtype, seed=0, state=True, lens=None, one=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    unit = lambda x: x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)  # noqa: E731
    lead = (B,) if one else (B, T)
    x = dict(q=unit(_rand(gen, *lead, Hk, dk)).to(dtype), k=unit(_rand(gen, *lead, Hk, dk)).to(dtype),
             v=_rand(gen, *lead, H, dv).to(dtype),
             g=-torch.exp2(-9.0 * torch.rand(H, generator=gen, device="cuda")), scale=dk ** -0.5,
             S0=_rand(gen, B, H, dk, dv) if state else None,
             lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"))
    return x, gen


def absolute(x):
    return {n: v.abs() if isinstance(v, torch.Tensor) and n not in ("g", "lens") else v for n, v in x.items()}


def fwd_ref(x):
    a = absolute(x)
    arg = ("q", "k", "v", "g", "scale", "S0", "lens")
    return ref.prefill(*(x[n] for n in arg))[:2], ref.prefill(*(a[n] for n in arg))[:2]


def terms(*sizes):
    """fp32 sums of that many terms, and weights exp(g n) good to about 2^-24 |g n|
    where they matter (|g n| < 100)."""
    return sum(sizes) + 256


def check_prefill(x, o, S_T):
    """bf16: the weight of each pair and the state are rounded to bf16 once, each on
    its own part of the sum: one rounding on the magnitude.  S_T: fp32 throughout."""
    (o_ref, S_ref), (o_mag, S_mag) = fwd_ref(x)
    dt = x["q"].dtype
    T = x["v"].shape[1]
    n = terms(2 * T, x["q"].shape[-1])
    ref.check("o", o, o_ref, o_mag, dt, 1 if dt == BF else 0, n)
    if S_T is not None:
        ref.check("S_T", S_T, S_ref, S_mag, dt, 0, n)


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
    say("prefill", size, dtype)
    x, _ = make(*size, dtype, seed=size[1], state=size[1] % 2 == 1)
    o, S_T = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["scale"], x["S0"])
    torch.cuda.synchronize()
    check_prefill(x, o, S_T)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_lengths_leave_the_rest_alone(dtype):
    """Odd lengths, 0, 1, and values outside [0, T]; rows past them hold NaN and
    are neither read nor written."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    lens = [0, 1, 150, 97, -3, 999, 32, 33]
    B, T = len(lens), 150
    x, _ = make(B, T, 4, 2, 64, 128, dtype, seed=5, lens=lens)
    clean = {n: x[n].clone() for n in "qkv"}
    for b, n in enumerate(ref.lengths(lens, B, T)):
        for t in "qkv":
            x[t][b, n:] = float("nan")
            clean[t][b, n:] = 0
    o = torch.full((B, T, 4, 128), 7.0, dtype=dtype, device="cuda")
    _, S_T = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["scale"], x["S0"], x["lens"], o=o)
    torch.cuda.synchronize()
    for b, n in enumerate(ref.lengths(lens, B, T)):
        assert (o[b, n:] == 7.0).all()
        o[b, n:] = 0
    check_prefill({**x, **clean}, o, S_T)
    assert torch.equal(S_T[0], x["S0"][0]) and torch.equal(S_T[4], x["S0"][4])
    o2, _ = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["scale"], x["S0"], x["lens"])
    assert torch.equal(o2, o)                       # an allocated o is zero there


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_decays_at_their_ends(dtype):
    """No decay, a total one (also -infinity), a fast one, a slow one."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, _ = make(1, 130, 6, 6, 64, 64, dtype, seed=6)
    x["g"] = torch.tensor([0.0, float("-inf"), -1e30, -30.0, -1e-6, -0.5], device="cuda")
    o, S_T = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["scale"], x["S0"])
    torch.cuda.synchronize()
    check_prefill(x, o, S_T)
    dO, dS = torch.randn_like(x["v"]), torch.randn_like(x["S0"])
    got = kda.linear_backward(x["q"], x["k"], x["v"], x["g"], dO, x["scale"], x["S0"], dS)
    torch.cuda.synchronize()
    check_backward({**x, "dO": dO, "dS_T": dS}, got)


def test_prefill_in_place_state_and_continuation():
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, _ = make(2, 90, 2, 2, 128, 128, F32, seed=7)
    S = x["S0"].clone()
    o = torch.empty_like(x["v"])
    for lo, hi in ((0, 37), (37, 38), (38, 90)):
        part = [x[n][:, lo:hi].contiguous() for n in "qkv"]
        po = torch.empty_like(part[2])
        ws = torch.empty(max(1, kda.kda_linear_prefill_workspace_bytes(2, hi - lo, 2, 2, 128, 128, F32)),
                         dtype=torch.uint8, device="cuda")
        kda.kda_linear_prefill(*part, x["g"], x["scale"], S, po, S, workspace=ws)
        o[:, lo:hi] = po
    torch.cuda.synchronize()
    check_prefill(x, o, S)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_in_place_state_of_long_sequences(dtype):
    """Segments of one sequence run side by side; the final state may take the
    initial one's place all the same."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, _ = make(3, 2100, 2, 1, 64, 128, dtype, seed=17, lens=[2100, 700, 31])
    args = (x["q"], x["k"], x["v"], x["g"], x["scale"])
    o, S_T = kda.linear_prefill(*args, x["S0"], x["lens"])
    ws = torch.empty(kda.kda_linear_prefill_workspace_bytes(3, 2100, 2, 1, 64, 128, dtype), dtype=torch.uint8,
                     device="cuda")
    for _ in range(5):
        S, o2 = x["S0"].clone(), torch.zeros_like(o)
        kda.kda_linear_prefill(*args, S, o2, S, x["lens"], ws)
        torch.cuda.synchronize()
        assert torch.equal(S, S_T) and torch.equal(o2, o)


def test_long_slow_decays_keep_their_factor():
    """20,000 steps at decays near 1: the state's error stays that of fp32 sums.  Each of
    625 chunk updates rounds the state by at most 2^-24 of itself, at random: about
    sqrt(625) 2^-25 = 7.5e-7 of its norm, to which the weights add a few 2^-24; 4e-6
    leaves a factor of four.  A factor a^32 rounded once and multiplied 625 times would
    be off by up to 625 2^-25 = 1.9e-5."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, _ = make(1, 20000, 4, 4, 32, 32, F32, seed=18)
    x["g"] = torch.tensor([-1e-6, -3.1e-5, -1.7e-4, 0.0], device="cuda")
    _, S_T = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["scale"], x["S0"])
    torch.cuda.synchronize()
    a = torch.exp(x["g"].double())[:, None, None]
    S = x["S0"][0].double()
    for t in range(20000):
        S = a * S + x["k"][0, t].double()[:, :, None] * x["v"][0, t].double()[:, None]
    err = torch.linalg.vector_norm(S_T[0].double() - S, dim=(1, 2)) / torch.linalg.vector_norm(S, dim=(1, 2))
    assert (err < 4e-6).all(), err


def test_tensors_past_32_bit_offsets():
    """More than 2^31 elements a tensor: the last tokens against the same tokens alone,
    whose state is what the 4,096 before them leave (a^4096 < e^-200)."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    T, H, d, tail = 530000, 32, 128, 4160
    assert T * H * d > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(19)
    x = {n: torch.empty(1, T, H, d, dtype=BF, device="cuda").normal_(generator=gen) for n in "qkv"}
    g = torch.full((H,), -0.05, device="cuda")
    o, S_T = kda.linear_prefill(x["q"], x["k"], x["v"], g, 0.01)
    end = {n: x[n][:, -tail:].contiguous() for n in "qkv"}
    oe, Se = kda.linear_prefill(end["q"], end["k"], end["v"], g, 0.01)
    torch.cuda.synchronize()
    # both are the same sums in another order: rounding of the operands and the output
    mag = kda.linear_prefill(end["q"].abs(), end["k"].abs(), end["v"].abs(), g, 0.01)
    for a, b, m, tol in ((o[:, -64:], oe[:, -64:], mag[0][:, -64:], 2.0 ** -6), (S_T, Se, mag[1], 2.0 ** -14)):
        assert ((a.double() - b.double()).abs() <= tol * m.double()).all()
    del o, oe, mag, end
    # gradients reach the first tokens from the end: the same on the first ones alone
    dO = x["v"]
    got = kda.linear_backward(x["q"], x["k"], x["v"], g, dO, 0.01, want_dS0=False)
    head = {n: x[n][:, :tail].contiguous() for n in "qkv"}
    want = kda.linear_backward(head["q"], head["k"], head["v"], g, head["v"], 0.01, want_dS0=False)
    head = {n: t.abs() for n, t in head.items()}
    mag = kda.linear_backward(head["q"], head["k"], head["v"], g, head["v"], 0.01, want_dS0=False)
    torch.cuda.synchronize()
    for n in ("dq", "dk", "dv"):
        a, b, m = got[n][:, :64].double(), want[n][:, :64].double(), mag[n][:, :64].double()
        assert ((a - b).abs() <= 2.0 ** -6 * m).all(), n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_calls_on_a_given_stream(dtype):
    """stream= as a torch stream and as its handle, with another one current."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, gen = make(2, 700, 4, 2, 64, 64, dtype, seed=20)
    dO = _rand(gen, *x["v"].shape).to(dtype)
    args = (x["q"], x["k"], x["v"], x["g"])
    want = [*kda.linear_prefill(*args, x["scale"], x["S0"]), *kda.linear_backward(*args, dO, x["scale"]).values()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = [*kda.linear_prefill(*args, x["scale"], x["S0"], stream=stream),
               *kda.linear_backward(*args, dO, x["scale"], stream=stream).values()]
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def bwd_ref(x):
    a = absolute(x)
    arg = ("q", "k", "v", "g", "scale", "dO", "S0", "dS_T", "lens")
    return ref.backward(*(x[n] for n in arg)), ref.backward(*(a[n] for n in arg))


def check_backward(x, got):
    want, mag = bwd_ref(x)
    dt = x["q"].dtype
    B, T, H, dv = x["v"].shape
    n = terms(2 * T, max(dv, x["q"].shape[-1]), H // x["q"].shape[2])
    for name in ("dq", "dk", "dv", "dS0"):
        # as in check_prefill: one rounding on each part; dS0 is fp32 throughout
        ref.check(name, got[name], want[name], mag[name], dt, 1 if dt == BF and name != "dS0" else 0, n)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", SIZES[:-2] + [(1, 410, 2, 1, 128, 128)])
def test_backward(size, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("backward", size, dtype)
    state = size[1] % 2 == 0
    x, gen = make(*size, dtype, seed=100 + size[1], state=state)
    x["dO"] = _rand(gen, *x["v"].shape).to(dtype)
    x["dS_T"] = _rand(gen, size[0], size[2], size[4], size[5]) if state else None
    got = kda.linear_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], x["scale"], x["S0"], x["dS_T"])
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
    clean = {n: x[n].clone() for n in ("q", "k", "v", "dO")}
    for b, n in enumerate(ref.lengths(lens, B, T)):
        for t in clean:
            x[t][b, n:] = float("nan")
            clean[t][b, n:] = 0
    out = {n: torch.full_like(x[n[1:]], 7.0) for n in ("dq", "dk", "dv")}
    got = kda.linear_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], x["scale"], x["S0"], x["dS_T"],
                              x["lens"], **out)
    torch.cuda.synchronize()
    for b, n in enumerate(ref.lengths(lens, B, T)):
        for t in out.values():
            assert (t[b, n:] == 7.0).all()
            t[b, n:] = 0
    check_backward({**x, **clean}, got)
    assert torch.equal(got["dS0"][0], x["dS_T"][0])


def test_backward_against_differences_of_the_forward_call():
    """The loss is linear in q, in k, in v and in S0 alone, so a difference of any
    width is exact up to fp32 rounding: both sides are sums of at most
    T dk dv terms in fp32, near 2^-24 sqrt(terms) of their magnitude; 1e-4 of
    the loss's magnitude leaves a factor of ten."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, gen = make(2, 75, 4, 2, 64, 32, F32, seed=9)
    dO, dS = _rand(gen, *x["v"].shape), _rand(gen, 2, 4, 64, 32)

    def loss(y):
        o, S = kda.linear_prefill(y["q"], y["k"], y["v"], y["g"], y["scale"], y["S0"])
        return float((o.double() * dO).sum() + (S.double() * dS).sum())

    got = kda.linear_backward(x["q"], x["k"], x["v"], x["g"], dO, x["scale"], x["S0"], dS)
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("S0", "dS0")):
        way = _rand(gen, *x[name].shape)
        up, down = loss({**x, name: x[name] + way}), loss({**x, name: x[name] - way})
        want = float((got[key].double() * way).sum())
        assert abs((up - down) / 2 - want) < 1e-4 * max(1.0, abs(up), abs(down)), (name, up, down, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [(1, 1, 1, 32, 32), (3, 2, 1, 64, 128), (2, 4, 4, 128, 128), (5, 3, 3, 128, 32),
                                  (2, 6, 2, 32, 64), (40, 32, 32, 128, 128)])
def test_decode(size, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    B, H, Hk, dk, dv = size
    x, _ = make(B, 1, H, Hk, dk, dv, dtype, seed=B, one=True)
    x["g"][0] = float("-inf")
    S = x["S0"].clone()
    o = kda.linear_decode_step(x["q"], x["k"], x["v"], x["g"], S, x["scale"])
    torch.cuda.synchronize()
    a = absolute(x)
    arg = ("q", "k", "v", "g", "scale", "S0")
    for name, got, want, mag in zip(("o", "S"), (o, S), ref.decode(*(x[n] for n in arg)),
                                    ref.decode(*(a[n] for n in arg))):
        ref.check(name, got, want, mag, dtype, 0, terms(dk))


def _tree(gen, B, T, absent=True):
    t = torch.arange(T, device="cuda")
    back = 1 + (5 * torch.rand(B, T, generator=gen, device="cuda")).long()
    p = torch.clamp(t - back, min=-1).to(torch.int32)
    if absent and T > 3:
        p[0, T // 2] = -2                  # absent, with whatever hangs on it
        p[-1, T // 3] = T // 3             # itself: absent
        p[-1, T - 1] = 1 << 30
    return p


def check_tree(x, parent, o):
    dt, T = x["q"].dtype, x["v"].shape[1]
    a = absolute(x)
    arg = ("q", "k", "v", "g", "scale", "S0")
    ref.check("tree o", o, ref.tree(*(x[n] for n in arg), parent), ref.tree(*(a[n] for n in arg), parent), dt,
              1 if dt == BF else 0, terms(T, x["q"].shape[-1]))


TREES = [(1, 1, 1, 1, 32, 32), (2, 13, 4, 2, 64, 128), (3, 16, 2, 2, 128, 128), (2, 17, 3, 1, 128, 32),
         (2, 33, 2, 2, 32, 64), (2, 64, 4, 4, 128, 128), (1, 64, 2, 1, 64, 64), (1, 49, 2, 2, 128, 64)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", TREES)
def test_tree_and_commit(size, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("tree", size, dtype)
    B, T, H, Hk, dk, dv = size
    x, gen = make(*size, dtype, seed=T)
    parent = _tree(gen, B, T)
    o = kda.linear_tree(x["q"], x["k"], x["v"], x["g"], x["S0"], parent, x["scale"])
    torch.cuda.synchronize()
    check_tree(x, parent, o)
    a = absolute(x)
    for shift in (0, 1, 2, T // 2, T - 1, T):
        accepted = ((torch.arange(B, device="cuda") * 3 + shift) % (T + 1) - 1).to(torch.int32)
        out = torch.full_like(x["S0"], 7.0)
        kda.linear_tree_commit(x["k"], x["v"], x["g"], x["S0"], parent, accepted, S_out=out)
        S = x["S0"].clone()
        kda.linear_tree_commit(x["k"], x["v"], x["g"], S, parent, accepted)       # in place
        torch.cuda.synchronize()
        sevens = torch.full_like(out, 7.0)
        want = ref.commit(x["k"], x["v"], x["g"], x["S0"], parent, accepted, sevens)
        mag = ref.commit(a["k"], a["v"], a["g"], a["S0"], parent, accepted, sevens)
        ref.check("S_out", out, want, mag, dtype, 0, terms(T))
        for b in range(B):
            if (out[b] == 7.0).all():
                assert torch.equal(S[b], x["S0"][b])                              # skipped
            else:
                assert torch.equal(S[b], out[b])
            if accepted[b] == -1:
                assert torch.equal(out[b], x["S0"][b])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_shapes_and_bad_values(dtype):
    """A chain, a star, nothing at all, parents and accepted nodes out of range, a
    total decay."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    T = 64
    x, _ = make(4, T, 2, 2, 128, 128, dtype, seed=11)
    x["g"] = torch.tensor([float("-inf"), -0.02], device="cuda")
    t = torch.arange(T, dtype=torch.int32, device="cuda")
    parent = torch.stack([t - 1, torch.full_like(t, -1), torch.full_like(t, -5), T - t])
    x["q"][2] = float("nan")               # all absent: nothing of it is used
    clean = {n: x[n].clone() for n in x if isinstance(x[n], torch.Tensor)}
    clean["q"][2] = 0
    o = kda.linear_tree(x["q"], x["k"], x["v"], x["g"], x["S0"], parent, x["scale"])
    out = torch.full_like(x["S0"], 7.0)
    accepted = torch.tensor([T, -2, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    kda.linear_tree_commit(x["k"], x["v"], x["g"], x["S0"], parent, accepted, S_out=out)
    torch.cuda.synchronize()
    assert (out == 7.0).all()
    assert (o[2] == 0).all()
    check_tree({**x, **clean}, parent, o)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_paged_calls_equal_the_dense_ones(dtype):
    """Pool rows in any order, a row shared by two readers, slots out of range."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    B, T, H, Hk, dk, dv = 4, 70, 4, 2, 64, 128
    x, gen = make(B, T, H, Hk, dk, dv, dtype, seed=12, lens=[70, 0, 33, 5])
    pool = _rand(gen, 9, H, dk, dv)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (x["q"], x["k"], x["v"], x["g"], x["scale"])
    nbytes = kda.kda_linear_prefill_workspace_bytes(B, T, H, Hk, dk, dv, dtype)
    ws = torch.empty(max(1, nbytes), dtype=torch.uint8, device="cuda")

    def rows(t, slots, src):
        return torch.stack([t[s] if 0 <= s < 9 else src for s in slots])

    # prefill: sequence 2 has no row to read, so nothing of it is written
    p, slots_in, slots_out = pool.clone(), i32(3, 3, 9, 0), i32(5, 1, 2, 0)
    o = torch.full_like(x["v"], 7.0)
    kda.kda_linear_prefill_paged(*args, p, slots_in, slots_out, o, x["lens"], ws)
    S0 = rows(pool, slots_in.tolist(), pool[0])
    od, Sd = kda.linear_prefill(*args, S0, x["lens"], o=torch.full_like(x["v"], 7.0))
    want = pool.clone()
    for b in (0, 1, 3):
        want[int(slots_out[b])] = Sd[b]
    od[2] = 7.0
    assert torch.equal(o, od) and torch.equal(p, want)
    # no tables: zero states in, none out
    p = pool.clone()
    kda.kda_linear_prefill_paged(*args, p, None, None, o, None, ws)
    od, _ = kda.linear_prefill(*args)
    assert torch.equal(o, od) and torch.equal(p, pool)
    # decode
    q, k, v = (x[n][:, 0].contiguous() for n in "qkv")
    p, slots = pool.clone(), i32(8, -1, 0, 4)
    o = torch.full_like(v, 7.0)
    kda.kda_linear_decode_step_paged(q, k, v, x["g"], x["scale"], p, slots, o)
    S = rows(pool, slots.tolist(), pool[0])
    od = kda.linear_decode_step(q, k, v, x["g"], S, x["scale"])
    want = pool.clone()
    for b in (0, 2, 3):
        want[int(slots[b])] = S[b]
    od[1] = 7.0
    assert torch.equal(o, od) and torch.equal(p, want)
    # tree and commit (T = 64 of the tokens)
    part = [x[n][:, :64].contiguous() for n in "qkv"]
    parent = _tree(gen, B, 64)
    slots = i32(6, 2, 100, 6)
    o = torch.full_like(part[2], 7.0)
    kda.kda_linear_tree_paged(*part, x["g"], x["scale"], pool, slots, parent, o)
    S = rows(pool, slots.tolist(), pool[0])
    od = kda.linear_tree(*part, x["g"], S, parent, x["scale"])
    od[2] = 7.0
    assert torch.equal(o, od)
    p, slots_out, accepted = pool.clone(), i32(6, 7, 1, -4), i32(20, 31, 3, 4)
    kda.kda_linear_tree_commit_paged(part[1], part[2], x["g"], parent, accepted, p, slots, slots_out)
    Sd = kda.linear_tree_commit(part[1], part[2], x["g"], S, parent, accepted, S_out=S.clone())
    want = pool.clone()
    want[6], want[7] = Sd[0], Sd[1]
    assert torch.equal(p, want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_chain_of_drafts_is_a_prefill(dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, _ = make(2, 40, 4, 4, 128, 128, dtype, seed=13)
    parent = (torch.arange(40, device="cuda") - 1).to(torch.int32).expand(2, 40).contiguous()
    o = kda.linear_tree(x["q"], x["k"], x["v"], x["g"], x["S0"], parent, x["scale"])
    S = kda.linear_tree_commit(x["k"], x["v"], x["g"], x["S0"].clone(), parent,
                               torch.full((2,), 39, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    check_prefill(x, o, S)


def test_serving_run_of_the_calls_together():
    """Norm and rotation, prompt, draft tree, commit, single tokens, on a side stream
    and with states in a pool; against the recurrence over the tokens that stay."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    B, T, H, Hk, d = 2, 45, 4, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(14)
    n_tok = T + 8 + 2
    raw = {n: _rand(gen, B, n_tok, h, d) for n, h in (("q", Hk), ("k", Hk), ("v", H))}
    g = torch.tensor([-0.5, -0.1, -0.02, 0.0], device="cuda")
    pos = torch.arange(n_tok, device="cuda", dtype=torch.int32).expand(B, n_tok).contiguous()
    freq = 10000.0 ** (-torch.arange(0, d, 2, device="cuda") / d)
    pool, slots = _rand(gen, 3, H, d, d), torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    pool0 = pool.clone()
    parent = torch.tensor([[-1, 0, 0, 1, 2, 3, 4, 5]] * B, dtype=torch.int32, device="cuda")
    accepted = torch.tensor([5, 4], dtype=torch.int32, device="cuda")     # paths 0 1 3 5 and 0 2 4
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        q, k = kda.qk_norm_rope(raw["q"], raw["k"], pos, freq, norm="l2")
        cut = lambda lo, hi: [x[:, lo:hi].contiguous() for x in (q, k, raw["v"])]  # noqa: E731
        a, b = cut(0, T), cut(T, T + 8)
        o1 = torch.empty_like(a[2])
        ws = torch.empty(max(1, kda.kda_linear_prefill_workspace_bytes(B, T, H, Hk, d, d, F32)), dtype=torch.uint8,
                         device="cuda")
        kda.kda_linear_prefill_paged(*a, g, 1.0, pool, slots, slots, o1, None, ws)
        o2 = torch.empty_like(b[2])
        kda.kda_linear_tree_paged(*b, g, 1.0, pool, slots, parent, o2)
        kda.kda_linear_tree_commit_paged(b[1], b[2], g, parent, accepted, pool, slots, slots)
        o3 = []
        for t in range(T + 8, n_tok):
            c = [x[:, t].contiguous() for x in (q, k, raw["v"])]
            o3.append(torch.empty_like(c[2]))
            kda.kda_linear_decode_step_paged(*c, g, 1.0, pool, slots, o3[-1])
    s.synchronize()
    assert torch.equal(pool[1], pool0[1])
    for i, path in enumerate(([0, 1, 3, 5], [0, 2, 4])):
        keep = list(range(T)) + [T + p for p in path] + [T + 8, T + 9]
        x = dict(q=q[i:i + 1, keep], k=k[i:i + 1, keep], v=raw["v"][i:i + 1, keep], g=g, scale=1.0,
                 S0=pool0[int(slots[i])][None], lens=None)
        o = torch.cat([o1[i], o2[i, path], *(y[i:i + 1] for y in o3)])[None]
        check_prefill(x, o, pool[int(slots[i])][None])


def test_captured_calls_replay():
    """Prompt, gradients, tree, commit and single token in one captured graph, replayed
    over changed inputs with eager work between."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    B, T, H, Hk, d = 2, 200, 4, 2, 64
    x, gen = make(B, T, H, Hk, d, d, BF, seed=15)
    dO, dS = _rand(gen, *x["v"].shape).to(BF), _rand(gen, B, H, d, d)
    parent = _tree(gen, B, 50)
    accepted = torch.tensor([20, 3], dtype=torch.int32, device="cuda")

    def work(x, S):
        o, S_T = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["scale"], x["S0"])
        gr = kda.linear_backward(x["q"], x["k"], x["v"], x["g"], dO, x["scale"], x["S0"], dS)
        p = [x[n][:, :50].contiguous() for n in "qkv"]
        ot = kda.linear_tree(*p, x["g"], S_T, parent, x["scale"])
        S.copy_(S_T)
        kda.linear_tree_commit(p[1], p[2], x["g"], S, parent, accepted)
        one = [x[n][:, 0].contiguous() for n in "qkv"]
        od = kda.linear_decode_step(*one, x["g"], S, x["scale"])
        return [o, S_T, ot, od, S, *gr.values()]

    S, Se = torch.empty_like(x["S0"]), torch.empty_like(x["S0"])
    work(x, S)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work(x, S)
    for i in range(4):
        for n in "qkv":
            x[n].copy_(_rand(gen, *x[n].shape) * 0.1)
        x["S0"].mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, work(x, Se)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_calls_repeat_bit_for_bit(dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    x, gen = make(2, 700, 4, 2, 128, 128, dtype, seed=16)
    dO = _rand(gen, *x["v"].shape).to(dtype)
    run = lambda: [*kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["scale"], x["S0"]),  # noqa: E731
                   *kda.linear_backward(x["q"], x["k"], x["v"], x["g"], dO, x["scale"], x["S0"]).values()]
    first = run()
    for _ in range(3):
        for a, b in zip(first, run()):
            assert torch.equal(a, b)


def test_the_most_sequences():
    """2^22 sequences of one token, from no state: o = scale (q . k) v, dq = scale (v . dO) k,
    dk = scale (v . dO) q, dv = scale (q . k) dO, and the same as a tree of one node over one slot
    of zeros.  Inputs are small integers with d = 32, so every product and sum is exact and only
    the output's rounding is left, at most half a step of bf16; of a tree, whose pair weight is
    one bf16 value for so many sequences, that weight's rounding too (and the two's product)."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("2^22 sequences")
    B, d, scale = 1 << 22, 32, 0.25
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v, dO = (torch.randint(-4, 5, (B, 1, 1, d), generator=gen, device="cuda").to(BF) for _ in range(4))
    g = torch.zeros(1, device="cuda")
    o, _ = kda.linear_prefill(q, k, v, g, scale, want_state=False)
    grads = kda.linear_backward(q, k, v, g, dO, scale, want_dS0=False)
    tree = torch.empty_like(v)
    kda.kda_linear_tree_paged(q, k, v, g, scale, torch.zeros(1, 1, d, d, device="cuda"),
                                     torch.zeros(B, dtype=torch.int32, device="cuda"),
                                     torch.full((B, 1), -1, dtype=torch.int32, device="cuda"), tree)
    qk = scale * (q.float() * k.float()).sum(-1, keepdim=True)
    vo = scale * (v.float() * dO.float()).sum(-1, keepdim=True)
    half = torch.finfo(BF).eps / 2
    for name, got, want, tol in (("o", o, qk * v.float(), half), ("tree", tree, qk * v.float(), 2 * half + half ** 2),
                                 ("dq", grads["dq"], vo * k.float(), half), ("dk", grads["dk"], vo * q.float(), half),
                                 ("dv", grads["dv"], qk * dO.float(), half)):
        worst = ((got.float() - want).abs() - want.abs() * tol).max().item()
        assert worst <= 0, (name, worst)
