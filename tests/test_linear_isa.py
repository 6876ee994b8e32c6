"""ISA check (CPU, needs hipcc) of the linear-attention kernels: no MFMA takes
as srcC the result of an MFMA of a different shape issued shortly before it
(a chain that has read stale registers on gfx950; see test_isa_mfma_chains)."""
import os
import shutil
import subprocess

import pytest

from linear_attention_recurrence_05_amd import build as kbuild
from test_isa_mfma_chains import mixed_shape_chains

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not available")


@pytest.mark.parametrize("source", ["kda_linear.hip", "kda_linear_tree.hip"])
def test_kernels_have_no_mixed_shape_srcc_chain(tmp_path, source):
    asm = tmp_path / "k.s"
    subprocess.run([os.environ.get("HIPCC", "hipcc"), *kbuild.source_flags(source), "--cuda-device-only", "-S",
                    os.path.join(kbuild.CSRC, source), "-o", str(asm)], check=True, capture_output=True)
    text = asm.read_text().split("\n")
    assert any("v_mfma_f32_16x16x32_bf16" in l for l in text)
    assert not any("v_pk_fma_f32" in l or "v_pk_mul_f32" in l or "v_pk_add_f32" in l for l in text)
    assert mixed_shape_chains(text) == []
