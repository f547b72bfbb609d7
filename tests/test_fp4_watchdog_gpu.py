"""Failure detection of the 4-bit products without a GPU fault: stage barriers
wait for bytes that never arrive (an inflated transaction count), every bounded
wait gives up after a short limit, the kernel unwinds and frees its TMEM, and
the host reads BWG_ERR_TIMEOUT.  The context stays usable: the next call is
exact."""
import numpy as np
import pytest
import torch

from test_fp4_gpu import dev, random_fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops


def stalled(ops, call):
    ops.set_watchdog_ns(50_000_000)  # 50 ms
    ops.debug_set_tx_extra(1024)
    try:
        call()
        st, word = ops.last_device_error()
    finally:
        ops.debug_set_tx_extra(0)
        ops.set_watchdog_ns(0)
    assert st == 5 and (word >> 56) == 1, (st, hex(word))


# few rows: a cluster on one tile's k-blocks, with one row tile and several; whole tiles, one and several a CTA;
# pairs with one and with two weight blocks
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("kernel,M,N,K", [(0, 16, 256, 4096), (0, 200, 300, 4096), (0, 40, 12000, 256), (0, 5, 40000, 512),
                                          (0, 1500, 2600, 2080), (1, 2001, 5003, 2080), (2, 2135, 7972, 3616)])
def test_dense_products_give_up(ops, kernel, M, N, K, fmt):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert ops.lib().bwg_fp4_kernel(M, N, K, 0, 0, sms) == kernel
    rng = np.random.default_rng(M)
    a, A = random_fp4(ops, M, K, fmt, rng, integers=True)
    b, B = random_fp4(ops, N, K, fmt, rng, integers=True)
    D = torch.zeros(M, N, device="cuda")
    stalled(ops, lambda: ops.gemm_fp4(a, b, out=D))
    ops.gemm_fp4(a, b, out=D)
    assert ops.last_device_error() == (0, 0)
    assert torch.equal(D.double(), dev(A) @ dev(B).t())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("N,swiglu", [(512, False), (512, True), (60, True)])
def test_grouped_products_give_up(ops, N, swiglu, fmt):
    off = np.array([0, 300, 300, 1000], np.int32)
    M, G, K = 1000, 3, 1056
    rng = np.random.default_rng(N)
    a, A = random_fp4(ops, M, K, fmt, rng, offsets=off, integers=True)
    b, B = random_fp4(ops, G * N, K, fmt, rng, groups=G, integers=True)
    n_out = N // 2 if swiglu else N
    D = torch.zeros(M, n_out, device="cuda")
    want = ops.grouped_gemm_fp4(a, b, swiglu=swiglu, out_dtype=torch.float32)
    stalled(ops, lambda: ops.grouped_gemm_fp4(a, b, swiglu=swiglu, out=D))
    ops.grouped_gemm_fp4(a, b, swiglu=swiglu, out=D)
    assert ops.last_device_error() == (0, 0)
    assert torch.equal(D, want)
    if not swiglu:
        for e in range(G):
            rows = slice(off[e], off[e + 1])
            assert torch.equal(D[rows].double(), dev(A[rows]) @ dev(B[e * N:(e + 1) * N]).t())


def test_a_call_behind_one_that_gives_up(ops):
    """A launch that set up while the stalled one ran starts after it."""
    rng = np.random.default_rng(3)
    a, A = random_fp4(ops, 16, 4096, "nvfp4", rng, integers=True)
    b, B = random_fp4(ops, 256, 4096, "nvfp4", rng, integers=True)
    D = torch.zeros(16, 256, device="cuda")
    y = torch.zeros(16, 256, device="cuda")

    def both():
        ops.gemm_fp4(a, b, out=D)
        ops.debug_set_tx_extra(0)
        ops.gemm_fp4(a, b, out=y)

    stalled(ops, both)
    assert torch.equal(y.double(), dev(A) @ dev(B).t())
