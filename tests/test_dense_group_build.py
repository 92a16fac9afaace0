"""What the compiler makes of the kernels that split a CTA's registers among its
warps (no GPU needed): the split adds up only with the registers a thread that
the source counts on, so another number fails here and not on the device."""
import os
import re
import shutil
import subprocess

import pytest

from compressed_sparse_long_c4a_gb300 import build as B


@pytest.mark.parametrize("source", ["dense_group.cu", "prompt_attn.cu"])
def test_registers_of_two_tile_kernels(tmp_path, source):
    if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("no nvcc")
    want = int(re.search(r"kStreamLaunchRegs = (\d+)", open(os.path.join(B.CSRC, "dense_stream.cuh")).read()).group(1))
    r = subprocess.run([B._nvcc(), *B.ARCH, *B.FLAGS, "-Xptxas", "-v", "-I", B.INCLUDE, "-I", B.CSRC, "-c", os.path.join(B.CSRC, source),
                        "-o", str(tmp_path / "x.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    for kernel in ("stream_attn_kernel", "dealt_attn_kernel"):
        found = re.findall(rf"entry function '\w*{kernel}ILi(\d+)E.*?Used (\d+) registers", r.stdout + r.stderr, re.S)
        assert sorted(int(d) for d, _ in found) == [64, 128, 192, 256]
        assert {int(n) for d, n in found if int(d) <= 128} == {want}
