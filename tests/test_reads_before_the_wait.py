"""A kernel that may start while the stream's earlier kernels run reads what they wrote only behind its own wait for
them (griddepcontrol.wait makes their memory visible; the order in which kernels start does not).  Checked on the
source: between the head of a kernel and its wait stands no call that reads global memory."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_moe_gather_gb300", "csrc")
READS = re.compile(r"__ldg\(|__ldcg\(|\bload1\(|\bload_raw\(|\bload8<|\bload_early\(|\bload_value\(|\bsequence\(|\bsequence_totals\(|"
                   r"\badd_slots\(|\btoken_factor\(|\bkeep_columns<|\bcount_chunks\(")


def kernels():
    """(file, head, text between the head and the wait) of every kernel with a wait."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(path) as f:
            text = f.read()
        for part in re.split(r"(?=__global__)", text)[1:]:
            body = part[part.index("{"):] if "{" in part else ""
            if "grid_dependency_wait()" in body:
                head = re.search(r"(\w+_kernel)\s*\(", part)
                yield os.path.basename(path), head and head.group(1), body[:body.index("grid_dependency_wait()")]


FOUND = [(f, h, b) for f, h, b in kernels() if f in ("balance.cu", "resnorm.cu", "resnorm_backward.cu", "mm_fp8.cuh")]


@pytest.mark.parametrize("file,head,before", FOUND, ids=[f"{f}:{h}" for f, h, _ in FOUND])
def test_nothing_is_read_before_the_wait(file, head, before):
    code = re.sub(r"//[^\n]*", "", before)
    assert not READS.search(code), f"{file}: {head} reads before its wait: {READS.search(code).group(0)}"


def test_the_kernels_were_found():
    assert {h for _, h, _ in FOUND} >= {"sum_parts_kernel", "balance_finish_kernel", "balance_kernel", "column_sums_kernel",
                                        "residual_norm_backward_kernel", "residual_norm_many_kernel", "mm_wide_kernel"}
