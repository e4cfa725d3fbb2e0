"""The wide kernels of products without an end keep their 128 sums a thread in registers: what an end needs is no part of
their arguments.  (With it the SwiGLU kernel spilled 24 bytes a thread, and 16384 rows over 128 experts took 83 us instead
of 80.5.)  Checked on what the assembler prints."""
import os
import re
import shutil
import subprocess

import pytest

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_moe_gather_gb300")


def test_plain_wide_products_do_not_spill(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    cmd = [nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "--expt-relaxed-constexpr", "-Xptxas", "-v", "-c", os.path.join(PKG, "csrc", "mm_fp8.cu"), "-o", str(tmp_path / "o")]
    log = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    spills = {name: int(stores) for name, stores in
              re.findall(r"Compiling entry function '(\S*mm_wide_kernel\S*)'.*?(\d+) bytes spill stores", log, re.S)}
    assert len(spills) == 2 and max(spills.values()) <= 4, spills
