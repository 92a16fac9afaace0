"""What the compiler makes of the dense chunk kernels (no GPU needed): the
split of a CTA's registers among its warps adds up only with the registers a
thread that the source counts on, so another number fails here and not on the
device."""
import os
import re
import shutil
import subprocess

import pytest

from compressed_sparse_long_c4a_gb300 import build as B


def test_registers_of_the_chunk_kernels(tmp_path):
    if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("no nvcc")
    src = os.path.join(B.CSRC, "dense_prefill.cu")
    fp8, bf16 = map(int, re.search(r"kLaunchRegs = kFp8 \? (\d+) : (\d+)", open(src).read()).groups())
    r = subprocess.run([B._nvcc(), *B.ARCH, *B.FLAGS, "-Xptxas", "-v", "-I", B.INCLUDE, "-I", B.CSRC, "-c", src, "-o", str(tmp_path / "x.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    found = re.findall(r"entry function '\w*dense_prefill_kernelILi(\d+)ELb([01])E.*?Used (\d+) registers", r.stdout + r.stderr, re.S)
    assert sorted((int(d), int(b), int(n)) for d, b, n in found) == [(64, 0, bf16), (64, 1, fp8), (128, 0, bf16), (128, 1, fp8)]
