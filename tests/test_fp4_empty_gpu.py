"""Grouped 4-bit products without columns to sum over (K = 0): zeros in the
groups' rows, nothing in the rows of no group."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,swiglu", [(48, False), (512, False), (512, True), (60, True)])
@pytest.mark.parametrize("offsets,bad", [([0, 3, 3, 7], False), ([0, 0, 0, 0], False), ([0, 4, 4, 12], False),
                                         ([0, 5, 2, 9], True), ([0, 4, 8, 40], True), ([0, 2, 5, -1], True),
                                         ([0] + [1] * 40 + [5], False)])
def test_no_columns(ops, offsets, bad, N, swiglu, dtype, fmt):
    """Broken offsets: every row below the largest of them, at most all."""
    M, G = 12, len(offsets) - 1
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    a = ops.quantize_fp4(torch.zeros(M, 0, device="cuda"), fmt, group_offsets=off)
    b = ops.quantize_fp4(torch.zeros(G, N, 0, device="cuda"), fmt)
    n_out = N // 2 if swiglu else N
    buf = torch.full((M, n_out + 3), 9.0, device="cuda", dtype=dtype)
    ops.grouped_gemm_fp4(a, b, swiglu=swiglu, out=buf[:, 1:1 + n_out])
    status, _ = ops.last_device_error()
    assert status == (1 if bad else 0)
    n = min(M, max(offsets))
    assert bool((buf[:n, 1:1 + n_out] == 0).all())
    assert bool((buf[n:] == 9).all()) and bool((buf[:, :1] == 9).all()) and bool((buf[:, 1 + n_out:] == 9).all())
