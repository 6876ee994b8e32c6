"""The gated norm and the norms between blocks on the GPU against their 64-bit definitions."""
import pytest
import torch

import delta_ref as ref
from gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
#: fp32 roundings on the way of one element beside its row's sums: the row's length, the gate, the
#: products.
STEPS = 64


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(gen, *s):
    return torch.randn(*s, generator=gen, device="cuda")


GATED = [((1,), 32), ((3, 5), 64), ((1, 1, 3), 128), ((257,), 32), ((2, 33, 3), 128), ((4, 1001, 2), 64),
         ((9000,), 128), ((40000,), 32)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("lead,d", GATED)
def test_gated_norm(lead, d, act, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("gated norm", lead, d, act, dtype)
    gen = _gen(d)
    x, dy = (_rand(gen, *lead, d).to(dtype) for _ in range(2))
    z = (4.0 * _rand(gen, *lead, d)).to(dtype)
    x[(0,) * len(lead)] = 0                                  # a row of zeros
    for w in (None, 1.0 + 0.2 * _rand(gen, d)):
        y = kda.gated_norm(x, z, w, act, 1e-5)
        got = kda.gated_norm_backward(x, z, w, dy, act, 1e-5)
        torch.cuda.synchronize()
        want = ref.gated_norm(x, z, w, act, 1e-5)
        ref.check_sums("y", y, want, want.abs(), STEPS + d)
        want, mag = ref.gated_norm_backward(x, z, w, dy, act, 1e-5)
        for n in ("dx", "dz", "dw"):
            if n == "dw" and w is None:
                assert got[n] is None
                continue
            ref.check_sums(n, got[n], want[n], mag[n], STEPS + d + (x.numel() // d if n == "dw" else 0))


def test_gated_norm_in_place():
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    gen = _gen(1)
    x, z, dy = (_rand(gen, 5000, 64).to(BF) for _ in range(3))
    w = _rand(gen, 64)
    want, grads = kda.gated_norm(x, z, w), kda.gated_norm_backward(x, z, w, dy)
    a, d, dz = x.clone(), dy.clone(), torch.empty_like(x)
    kda.kda_gated_norm(a, z, w, "silu", 1e-6, a)
    kda.kda_gated_norm_backward(x, z, w, "silu", 1e-6, d, d, dz, None)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(d, grads["dx"]) and torch.equal(dz, grads["dz"])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gates_at_their_ends_and_rows_out_of_range(dtype):
    """Gates far out saturate; rows whose squares leave fp32 keep their norm; an infinity or NaN
    stays in its row."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    gen = _gen(2)
    x, z, dy = _rand(gen, 64, 128), _rand(gen, 64, 128), _rand(gen, 64, 128)
    z[0], z[1], z[2], z[3] = 200.0, -200.0, 60.0, -60.0
    for i, s in enumerate((1e30, 1e-25, 1e36, 1e-36, 3e19, 1e-18)):
        x[8 + i] *= s
    x, z, dy = (t.to(dtype) for t in (x, z, dy))
    bad = x.clone()
    bad[20, 3], bad[30, 5] = float("inf"), float("nan")
    for act in ("silu", "sigmoid"):
        y, yb = kda.gated_norm(x, z, None, act, 1e-30), kda.gated_norm(bad, z, None, act, 1e-30)
        got = kda.gated_norm_backward(x, z, None, dy, act, 1e-30)
        gb = kda.gated_norm_backward(bad, z, None, dy, act, 1e-30)
        torch.cuda.synchronize()
        want = ref.gated_norm(x, z, None, act, 1e-30)
        ref.check_sums("y", y, want, want.abs(), STEPS + 128)
        want, mag = ref.gated_norm_backward(x, z, None, dy, act, 1e-30)
        for n in ("dx", "dz"):
            # beyond bf16's and fp32's largest the gradient of a tiny row is infinite, as rounding gives it
            fits = want[n].abs() < 3e38
            ref.check_sums(n, torch.where(fits.cuda(), got[n], 0.0), torch.where(fits, want[n], 0.0), mag[n].clamp(max=1e300), STEPS + 128)
        rest = [i for i in range(64) if i not in (20, 30)]
        assert torch.equal(y[rest], yb[rest]) and torch.equal(got["dx"][rest], gb["dx"][rest])
        assert torch.equal(got["dz"][rest], gb["dz"][rest])


BLOCK = [(1, 8), (3, 64), (5, 520), (7, 2048), (2, 2056), (33, 4096), (300, 72), (2, 7168), (3, 8192), (2, 16384), (1300, 1024)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm_y", [True, False])
@pytest.mark.parametrize("rows,D", BLOCK)
def test_block_norm(rows, D, norm_y, dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("block norm", rows, D, norm_y, dtype)
    gen = _gen(D)
    y, r, dn, dh = (_rand(gen, rows, D).to(dtype) for _ in range(4))
    z = (3.0 * _rand(gen, rows, D)).to(dtype)
    w_y, w_n = 1.0 + 0.2 * _rand(gen, D), 1.0 + 0.2 * _rand(gen, D)
    kw = dict(norm_y=norm_y, scale=0.37, eps=1e-5)
    for gate, wy, wn in ((z, w_y, w_n), (None, None, None), (z, None, w_n), (None, w_y, None)):
        h, n = kda.block_norm(y, r, z=gate, w_y=wy, w_n=wn, **kw)
        want, mag = ref.block_norm(y, r, gate, wy, wn, **kw)
        grads = kda.block_norm_backward(y, h, dn, dh, z=gate, w_y=wy, w_n=wn, **kw)
        torch.cuda.synchronize()
        ref.check_sums("h", h, want["h"], mag["h"], STEPS + D)
        ref.check_sums("n", n, want["n"], mag["n"], STEPS + D)
        want, mag = ref.block_norm_backward(y, h, dn, dh, gate, wy, wn, **kw)
        for name, t in want.items():
            if t is None:
                assert grads[name] is None
            else:
                ref.check_sums(name, grads[name], t, mag[name], STEPS + 2 * D + (rows if name.startswith("dw") else 0))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_block_norm_without_a_block(dtype):
    """The first norm of a stack: of the stream alone; and gradients without dh."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    gen = _gen(3)
    r, dn, w = _rand(gen, 70, 1000).to(dtype), _rand(gen, 70, 1000).to(dtype), _rand(gen, 1000)
    h, n = kda.block_norm(None, r, w_n=w)
    got = kda.block_norm_backward(None, r, dn, w_n=w)
    inplace = r.clone()
    kda.kda_block_norm(None, None, None, inplace, w, False, 1.0, 1e-6, None, inplace)
    torch.cuda.synchronize()
    assert h is r and torch.equal(inplace, n)
    want, mag = ref.block_norm(None, r, None, None, w, False, 1.0, 1e-6)
    ref.check_sums("n", n, want["n"], want["n"].abs(), STEPS + 1000)
    want, mag = ref.block_norm_backward(None, r, dn, None, None, None, w, False, 1.0, 1e-6)
    ref.check_sums("dr", got["dr"], want["dr"], mag["dr"], STEPS + 1000)
    ref.check_sums("dw_n", got["dw_n"], want["dw_n"], mag["dw_n"], STEPS + 1070)
    assert got["dy"] is None and got["dz"] is None and got["dw_y"] is None


def test_block_norm_in_place():
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    gen = _gen(4)
    y, r, z, dn, dh = (_rand(gen, 600, 2048).to(BF) for _ in range(5))
    w = _rand(gen, 2048)
    h, n = kda.block_norm(y, r, z=z, w_y=w, w_n=w, norm_y=True)
    want = kda.block_norm_backward(y, h, dn, dh, z=z, w_y=w, w_n=w, norm_y=True)
    y1, r1, dr = y.clone(), r.clone(), dh.clone()
    kda.kda_block_norm(y1, z, w, r1, w, True, 1.0, 1e-6, r1, y1)
    dy, dz = torch.empty_like(y), torch.empty_like(y)
    kda.kda_block_norm_backward(y, z, w, h, w, True, 1.0, 1e-6, dn, dr, dr, dy, dz, None, None)
    torch.cuda.synchronize()
    assert torch.equal(r1, h) and torch.equal(y1, n)
    assert torch.equal(dr, want["dr"]) and torch.equal(dy, want["dy"]) and torch.equal(dz, want["dz"])


@pytest.mark.parametrize("D", [64, 4096])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_block_rows_out_of_range(dtype, D):
    """Rows of the stream and of the block's output whose squares leave fp32; an infinity or NaN
    stays in its row."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    gen = _gen(5)
    y, r, dn, dh = (_rand(gen, 24, D) for _ in range(4))
    for i, s in enumerate((1e30, 1e-25, 1e35, 1e-36)):
        y[2 + i] *= s
        r[8 + i] *= s
        y[8 + i] = 0
    y, r, dn, dh = (t.to(dtype) for t in (y, r, dn, dh))
    bad = r.clone()
    bad[15, 3], bad[20, 5] = float("inf"), float("nan")
    kw = dict(norm_y=True, eps=1e-30, scale=1.0)
    h, n = kda.block_norm(y, r, **kw)
    hb, nb = kda.block_norm(y, bad, **kw)
    got = kda.block_norm_backward(y, h, dn, dh, **kw)
    torch.cuda.synchronize()
    want, mag = ref.block_norm(y, r, None, None, None, **kw)
    ref.check_sums("h", h, want["h"], mag["h"], STEPS + D)
    ref.check_sums("n", n, want["n"], mag["n"], STEPS + D)
    want, mag = ref.block_norm_backward(y, h, dn, dh, None, None, None, **kw)
    for name in ("dr", "dy"):
        # dr of a tiny row is large, dy's magnitude with it: what fp32 holds is compared
        fits = (mag[name] < 1e37).all(-1, keepdim=True)
        assert fits.double().mean() > 0.7
        ref.check_sums(name, torch.where(fits.cuda(), got[name], 0.0), torch.where(fits, want[name], 0.0), mag[name].clamp(max=1e300), STEPS + 2 * D)
    rest = [i for i in range(24) if i not in (15, 20)]
    assert torch.equal(h[rest], hb[rest]) and torch.equal(n[rest], nb[rest])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norms_on_a_given_stream_and_in_a_graph(dtype):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    gen = _gen(6)
    x, z, dy = (_rand(gen, 900, 128).to(dtype) for _ in range(3))
    y, r, g, dn, dh = (_rand(gen, 90, 1280).to(dtype) for _ in range(5))
    w, wd = _rand(gen, 128), _rand(gen, 1280)

    def once(stream=None):
        h, n = kda.block_norm(y, r, z=g, w_y=wd, w_n=wd, norm_y=True, stream=stream)
        return [kda.gated_norm(x, z, w, stream=stream), *kda.gated_norm_backward(x, z, w, dy, stream=stream).values(), h, n,
                *kda.block_norm_backward(y, h, dn, dh, z=g, w_y=wd, w_n=wd, norm_y=True, stream=stream).values()]

    want = once()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = once(stream)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = once()
    for _ in range(4):
        for t in got:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        torch.ones(1000, device="cuda").sum().item()
