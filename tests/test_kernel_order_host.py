"""Memory order of the kernels, checked in their sources: a wrong order shows in results
rarely or never, so no run of a kernel can be relied on to find it."""
import os
import re

import dense_gemm_row_gb300

CSRC = os.path.join(os.path.dirname(dense_gemm_row_gb300.__file__), "csrc")


def sources():
    """(file name, text without comments) of every kernel source."""
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            with open(os.path.join(CSRC, name)) as f:
                yield name, re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_no_read_only_loads_in_kernels_that_overlap_their_predecessor():
    """The read-only path (__ldg, ld.global.nc) is for memory that stays as it is while
    the kernel runs. A kernel that starts as a programmatic dependent runs while its
    predecessor writes, and the wait for it orders ordinary loads only.

    gemm_tc_kernel.cuh's row_corr and col_corr are outside the rule: the kernels that
    write them do not release their dependents before they end."""
    found = []
    for name, text in sources():
        for m in re.finditer(r"__ldg\s*\(([^()]*)|ld\.global\.nc", text):
            if not re.match(r"p\.(row|col)_corr", m.group(1) or ""):
                found.append((name, m.group(0)))
    assert not found
    writers = [t for n, t in sources() if n == "gemm_tc_int.cu"]
    for kernel in ("u8_row_corr_kernel", "u8_col_corr_kernel"):
        body = re.search(kernel + r"\(const uint8_t.*?\n}\n", writers[0], flags=re.S).group(0)
        assert "grid_launch_dependents" not in body
