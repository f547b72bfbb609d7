"""Sources of the kernels that launch_behind starts while the work before them may
still be running: they wait for it before they touch global memory, and read what it
may have written with plain loads.  No GPU."""
import os
import re

from test_overlap_host import CSRC, code


def read(name):
    return code(os.path.join(CSRC, name))


def sources():
    names = [n for n in sorted(os.listdir(CSRC)) if n.endswith((".cu", ".cuh"))]
    return {n for n in names if re.search(r"\blaunch_(behind|pair_behind)\(", read(n))}


def test_there_are_such_sources():
    assert sources() == {"gemm_body.cuh", "gemm_gated.cu", "gemm_tn.cu", "gemm_small_m.cu"}


def test_they_read_with_plain_loads():
    for name in sources():
        for word in ("__ldg", "ld.global.nc", "__restrict__"):
            assert word not in read(name), "%s in %s" % (word, name)


def test_kernels_wait_before_they_read():
    """Every kernel of gemm_gated.cu and gemm_tn.cu is the shared body, in a form that
    waits, or waits itself; so does the gated form of the small-M kernel, before its
    first loads."""
    for name in ("gemm_gated.cu", "gemm_tn.cu"):
        for kernel in read(name).split("__global__")[1:]:
            body = kernel.split("{", 1)[1].strip()
            assert body.startswith("gemm_body<2, 1, ") or body.startswith("grid_dependency_wait();"), body[:80]
    small = read("gemm_small_m.cu")
    assert re.search(r"if constexpr \(SW\) \{\s*grid_dependency_wait\(\);", small)
    assert small.index("grid_dependency_wait();") < small.index("producer.issue(S, &aborted);")


def test_the_shared_body_waits():
    body = read("gemm_body.cuh")
    behind = body.index("constexpr bool kBehind = TN || EPI >= kEpiSwigluKeep || (SW && !GROUPED);")
    offsets = body.index("if constexpr (kBehind) grid_dependency_wait();", behind)
    assert offsets < body.index("grouped_tables_warp(p.group_offsets", behind)  # the warp that reads the offsets
    roles = body.index("if constexpr (kBehind) {\n    grid_dependency_wait();", offsets)
    assert roles < body.index("tma_load_", behind) and roles < body.index("emit = [&]", behind)


def test_dependents_are_let_in_after_the_kernels_own_tmem():
    """A kernel that allocates TMEM without a limit on its wait must hold it before it
    lets the kernel behind it become resident: that one could take it first, and then
    wait for this grid to end."""
    for name in sources():
        text = read(name)
        for kernel in re.split(r"__global__|__device__ void gemm_body", text)[1:]:
            alloc = [m.start() for m in re.finditer(r"\btmem_alloc<", kernel)]
            trigger = [m.start() for m in re.finditer(r"\bgrid_dependents_launch\(\)", kernel)]
            if not alloc or not trigger:
                continue
            assert len(alloc) == 1
            barrier = re.compile(r"\b(cluster_sync_all|__syncthreads)\(\)").search(kernel, alloc[0])
            assert barrier and barrier.start() < min(trigger), name
