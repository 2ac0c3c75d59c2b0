"""The kernels' shared headers, all of them in one translation unit."""
from __future__ import annotations

import glob
import os
import subprocess


def test_headers_together(tmp_path):
    from sparse_attention_kv_row_gb300 import build

    names = sorted(os.path.basename(p) for p in glob.glob(os.path.join(build.CSRC, "*.cuh")))
    assert len(names) > 5
    src = tmp_path / "all.cu"
    src.write_text("".join(f'#include "{n}"\n' for n in names))
    r = subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-I", build.CSRC, "-c", str(src), "-o",
                        str(tmp_path / "all.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
