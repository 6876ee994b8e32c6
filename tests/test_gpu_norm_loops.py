"""The gated norm and the norms between blocks over more rows than their launches have workgroups, in
every variant of threads and pieces a row, with the weights' gradients over all of them."""
import pytest
import torch

import delta_ref as ref
from gpu_common import need_gpu, say
from test_gpu_layer_norms import BF, F32, _gen, _rand

pytestmark = pytest.mark.gpu


def check_rows(name, got, want):
    """Each row in norm.  A bf16 rounding is at most 2^-8 of its element, so at most that of a row;
    what fp32 computes is off by a few tens of 2^-24 (1e-6 to 3e-6) of a row; a row that is another's, or
    was not written, is off by all of it."""
    got, want = got.double().cpu(), want.flatten(0, -2)
    off = (got.flatten(0, -2) - want).norm(dim=1) / want.norm(dim=1)
    limit = 2.0 ** -8 + 1e-5 if name[1] == BF else 1e-5
    assert off.max() < limit, (name, int(off.argmax()), float(off.max()))


def check_weight(name, got, want, rows):
    """A weight's gradient in norm: sums of `rows` terms of either sign.  Each is off by a few tens of
    2^-24, at random, and so are the partial sums: 1e-6 to 5e-6 of the norm.  A row left out is
    rows^(-1/2) of it."""
    off = float((got.double().cpu() - want).norm() / want.norm())
    assert off < 1e-5 < 0.1 * rows ** -0.5, (name, off)


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_gated_norm_loops(d, dtype, act):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    per = 256 // (d // (8 if dtype == BF else 4))            # rows of a workgroup, of which a launch has 2,048
    rows = 2048 * per * 5 // 2 + per // 2 + 1
    say("gated norm", rows, d, act, dtype)
    gen = _gen(d)
    x, z, dy = (_rand(gen, rows, d).to(dtype) for _ in range(3))
    w = 1.0 + 0.2 * _rand(gen, d)
    y, got = kda.gated_norm(x, z, w, act, 1e-5), kda.gated_norm_backward(x, z, w, dy, act, 1e-5)
    torch.cuda.synchronize()
    check_rows(("y", dtype), y, ref.gated_norm(x, z, w, act, 1e-5))
    want, _ = ref.gated_norm_backward(x, z, w, dy, act, 1e-5)
    for n in ("dx", "dz"):
        check_rows((n, dtype), got[n], want[n])
    check_weight("dw", got["dw"], want["dw"], rows)


# (bf16's width, fp32's, rows of a workgroup, workgroups of a launch at most) for 64 threads a row of one and
# two pieces, 256 of one and two, 512, and 1,024 of two and (fp32) four
VARIANTS = [(512, 256, 4, 1024), (1000, 504, 4, 1024), (2048, 1024, 1, 1024), (4096, 2048, 1, 1024), (8192, 4096, 1, 512),
            (12288, 8192, 1, 256), (16384, 16384, 1, 256)]


@pytest.mark.parametrize("norm_y", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("variant", VARIANTS)
def test_block_norm_loops(variant, dtype, norm_y):
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    D, rows = variant[0 if dtype == BF else 1], variant[2] * variant[3] * 9 // 4 + 3
    say("block norm", rows, D, norm_y, dtype)
    gen = _gen(D)
    y, r, z, dn, dh = (_rand(gen, rows, D).to(dtype) for _ in range(5))
    w_y, w_n = 1.0 + 0.2 * _rand(gen, D), 1.0 + 0.2 * _rand(gen, D)
    kw = dict(norm_y=norm_y, scale=0.37, eps=1e-5)
    h, n = kda.block_norm(y, r, z=z, w_y=w_y, w_n=w_n, **kw)
    got = kda.block_norm_backward(y, h, dn, dh, z=z, w_y=w_y, w_n=w_n, **kw)
    torch.cuda.synchronize()
    want, _ = ref.block_norm(y, r, z, w_y, w_n, **kw)
    check_rows(("h", dtype), h, want["h"])
    check_rows(("n", dtype), n, want["n"])
    want, _ = ref.block_norm_backward(y, h, dn, dh, z, w_y, w_n, **kw)
    for name in ("dr", "dy", "dz"):
        check_rows((name, dtype), got[name], want[name])
    for name in ("dw_y", "dw_n"):
        check_weight(name, got[name], want[name], rows)
    # without the weights' gradients, and dr in place of dh, the same rows
    dr, dy, dz = dh.clone(), torch.empty_like(y), torch.empty_like(y)
    kda.kda_block_norm_backward(y, z, w_y, h, w_n, norm_y, 0.37, 1e-5, dn, dr, dr, dy, dz, None, None)
    torch.cuda.synchronize()
    assert torch.equal(dr, got["dr"]) and torch.equal(dy, got["dy"]) and torch.equal(dz, got["dz"])
