"""Sources of the kernels that are launched to overlap the kernel before them."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "blackwell_tensor_core_gb300", "csrc")


def code(path):
    """The file without its comments."""
    with open(path, encoding="utf-8") as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def overlapped_sources():
    return [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if "launch_overlapped(" in code(p)]


def test_there_are_such_sources():
    assert {os.path.basename(p) for p in overlapped_sources()} == {"moe.cu", "gemm_fp4.cu"}


def test_overlapped_kernels_read_with_plain_loads():
    """ld.global.nc (__ldg, or what the compiler makes of const __restrict__)
    may be used on memory that nobody writes while the kernel runs; a kernel
    that starts before the one ahead of it has ended still sees its inputs
    written."""
    for path in overlapped_sources():
        for word in ("__ldg", "ld.global.nc", "__restrict__"):
            assert word not in code(path), "%s in %s" % (word, os.path.basename(path))


def test_overlapped_kernels_wait_before_they_read():
    """Every kernel of these files waits for the one ahead of it."""
    for path in overlapped_sources():
        for kernel in code(path).split("__global__")[1:]:
            assert "grid_dependency_wait();" in kernel, "%s: %s" % (os.path.basename(path), kernel[:80])
