"""The check of a kernel's registers before its launch, on a host without a GPU: a
program around the shared body's launch code with a stand-in for the runtime's query.

Kernels that split their registers with setmaxnreg wait for ever if they were launched
with fewer than the split hands out, so that each of them is asked for its own count."""
import subprocess

import pytest

from blackwell_tensor_core_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <cuda_runtime.h>

static int g_regs[3], g_asked;
template <class K>
cudaError_t fake_attributes(cudaFuncAttributes* a, K kernel);
#define cudaFuncGetAttributes fake_attributes
#include "gemm_body.cuh"

__global__ void enough(bwg::GemmParams) {}
__global__ void too_few(bwg::GemmParams) {}
__global__ void unknown(bwg::GemmParams) {}

template <class K>
cudaError_t fake_attributes(cudaFuncAttributes* a, K kernel) {
  ++g_asked;
  const void* p = reinterpret_cast<const void*>(kernel);
  if (p == reinterpret_cast<const void*>(unknown)) return cudaErrorInvalidDeviceFunction;
  a->numRegs = p == reinterpret_cast<const void*>(enough) ? bwg::kRegsLaunch2C : bwg::kRegsLaunch2C - 8;
  return cudaSuccess;
}

int main() {
  for (int turn = 0; turn < 3; ++turn) {
    printf("%d", bwg::two_consumer_regs_ok(enough));
    printf("%d", bwg::two_consumer_regs_ok(too_few));
    printf("%d ", bwg::two_consumer_regs_ok(unknown));
  }
  printf("%d\n", g_asked);
}
"""


@pytest.fixture(scope="module")
def answers(tmp_path_factory):
    d = tmp_path_factory.mktemp("registers")
    src, exe = d / "registers.cu", d / "registers"
    src.write_text(PROGRAM)
    subprocess.run([build.nvcc(), "-std=c++17", *build.ARCH, "-I", build.CSRC, "-diag-suppress=177", "-o", str(exe),
                    str(src)], check=True, capture_output=True, text=True, timeout=600)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout.split()


def test_every_kernel_has_its_own_answer(answers):
    assert answers[:3] == ["100"] * 3


def test_known_kernels_are_asked_once(answers):
    assert int(answers[3]) <= 2 + 3
