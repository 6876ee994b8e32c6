"""What the norm kernels' launches and registers come to (CPU, needs the built library and hipcc)."""
import os
import re
import shutil
import subprocess

import pytest
import torch

from linear_attention_recurrence_05_amd import build as kbuild

CUS = 256


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_block_norm_gradients_use_every_cu(dtype):
    """A workgroup leaves one partial gradient of both weights: as many as a device has CUs, of any width."""
    kda = pytest.importorskip("linear_attention_recurrence_05_amd")
    if not os.path.exists(kbuild.library_path()):
        pytest.skip("library not built")
    for D in (8, 256, 264, 504, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 12288, kda.KDA_MAX_NORM_WIDTH):
        groups = kda.kda_block_norm_backward_workspace_bytes(1 << 20, D, dtype) / (2 * D * 4)
        assert groups % CUS == 0 and groups >= CUS, (D, groups)


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not available")
@pytest.mark.parametrize("source", ["kda_block_norm.hip", "kda_gated_norm.hip"])
def test_no_kernel_spills(tmp_path, source):
    """Every variant, of any width and type, holds its row in registers (what the compiler reports)."""
    out = subprocess.run([os.environ.get("HIPCC", "hipcc"), *kbuild.source_flags(source), "-Rpass-analysis=kernel-resource-usage",
                          "--cuda-device-only", "-c", os.path.join(kbuild.CSRC, source), "-o", str(tmp_path / "k.o")],
                         check=True, capture_output=True, text=True).stderr
    names = re.findall(r"Function Name: (\S+)", out)
    spills = [int(n) for n in re.findall(r"VGPRs Spill: (\d+)", out)]
    scratch = [int(n) for n in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", out)]
    assert names and len(names) == len(spills) == len(scratch)
    assert not [n for n, a, b in zip(names, spills, scratch) if a or b]
