"""What the compiler says of the kernels that are to keep their rows in registers."""
from __future__ import annotations

import os
import re
import subprocess

from exact_tiled_attention_fa_gb300 import build as fa_build


def test_norm_and_rotation_kernels_do_not_spill(tmp_path):
    """Bound by bytes with 64 and 128 registers a thread: a spill is memory traffic of its own."""
    src = os.path.join(fa_build.CSRC, "fa_qk_rope.cu")
    r = subprocess.run([fa_build._nvcc(), *fa_build.ARCH, *fa_build.NVCC_FLAGS, "-Xptxas", "-v", "-I", fa_build.INCLUDE, "-c", src,
                        "-o", str(tmp_path / "rope.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    spills = re.findall(r"(\d+) bytes spill stores, (\d+) bytes spill loads", r.stderr)
    assert len(spills) >= 37  # 12 forward and cache forms, 24 gradient forms, the weights' sum
    assert set(spills) == {("0", "0")}, r.stderr
