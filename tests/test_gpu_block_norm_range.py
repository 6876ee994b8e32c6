"""The norms between blocks of blocks' outputs near fp32's largest, which weight, gate and scale bring
back into range."""
import pytest
import torch

import delta_ref as ref
from gpu_common import need_gpu, say
from test_gpu_layer_norms import BF, F32, STEPS, _gen, _rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate,weight,scale", [(-8.0, 4.0, 0.5), (8.0, 40.0, 0.025), (-8.0, 1000.0, 1.0), (None, 8.0, 0.0625)])
def test_large_outputs_of_a_block(gate, weight, scale, dtype):
    """y of 2e38: y w_y, and dy y w_y of the gate's gradient, are beyond fp32, what they come to is not."""
    need_gpu()
    import linear_attention_recurrence_05_amd as kda
    say("large y", gate, weight, scale, dtype)
    gen, rows, D = _gen(4), 4, 512
    y = (2e38 * (0.5 + 0.5 * torch.rand(rows, D, generator=gen, device="cuda"))).to(dtype)
    r, dn, dh = (_rand(gen, rows, D).to(dtype) for _ in range(3))
    z = None if gate is None else (gate + 0.1 * _rand(gen, rows, D)).to(dtype)
    w_y = weight * (1.0 + 0.01 * _rand(gen, D))
    kw = dict(norm_y=False, scale=scale, eps=1e-5)
    h, n = kda.block_norm(y, r, z=z, w_y=w_y, **kw)
    got = kda.block_norm_backward(y, h, dn, dh, z=z, w_y=w_y, **kw)
    torch.cuda.synchronize()
    want, mag = ref.block_norm(y, r, z, w_y, None, **kw)
    for name, t in (("h", h), ("n", n)):
        assert (want[name].abs() < 3.3e38).all() and torch.isfinite(t).all(), name
        ref.check_sums(name, t, want[name], mag[name], STEPS + D)
    want, mag = ref.block_norm_backward(y, h, dn, dh, z, w_y, None, **kw)
    for name, t in want.items():
        if t is not None:
            assert (t.abs() < 3.3e38).all() and torch.isfinite(got[name]).all(), name
            ref.check_sums(name, got[name], t, mag[name], STEPS + 2 * D + rows)
