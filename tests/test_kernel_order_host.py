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


def test_barriers_that_the_peer_signals_are_waited_for_at_cluster_scope():
    """The epilogue warps of both CTAs of a pair give an accumulator back on the leader's
    tmem_empty barrier (mapa to rank 0). A wait at CTA scope is not ordered behind the
    peer's arrival, and the MMAs that follow overwrite what the peer still reads."""
    waits = []
    for name, text in sources():
        if not re.search(r"mapa_shared\(smem_u32\(&sm\.tmem_empty\[buf\]\), 0\)", text):
            continue
        for m in re.finditer(r"(mbar_wait\w*(?:<\w+>)?)\(smem_u32\(&sm\.tmem_empty", text):
            before = text[:m.start()]
            # the branch of single CTAs, whose barrier no other one signals
            single = before.rstrip().endswith("got =") and "} else {" in before[-90:]
            waits.append((name, m.group(1), single))
    kernels = {"gemm_block_tile.cuh", "gemm_epi_tile.cuh", "gemm_tc_kernel.cuh"}
    assert {name for name, _, _ in waits} == kernels
    for name, wait, single in waits:
        assert single or wait in ("mbar_wait_lazy<true>", "mbar_wait_bounded_cluster"), (name, wait)
